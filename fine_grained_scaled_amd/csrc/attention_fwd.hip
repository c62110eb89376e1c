// attention_fwd.hip -- causal attention over packed sequences with grouped
// heads, forward, on gfx950.
//
// For token t of a sequence and query head h, over the tokens u <= t of the
// same sequence and the key head h / (H / Hk):
//   z[u] = scale * q[t] . k[u],  out[t] = sum_u softmax(z)[u] v[u],
//   lse[t] = log sum_u exp z[u].
// One pass over the keys with a running maximum m and sum l: scores, sums and
// the output accumulate in FP32; the probabilities are rounded to BF16 once,
// for the matrix product with v (each at most 2^-8 off, relative).
//
// A workgroup of 4 waves owns 128 query rows of one key head: HB query heads
// of its group times 128 / HB tokens, each wave 32 tokens of one head, so the
// heads that share keys share the staged tiles and a short sequence wastes
// at most 31 rows a head.  Tiles of 64 keys and values are staged in LDS, two
// deep, by copies that pass no register.  The scores are computed transposed,
// S^T = K Q^T, so a lane holds 32 keys of one query: its maximum and sum need
// one exchange between lane halves, and its probabilities are already the B
// operand of O^T = V^T P^T (attention_device.h).
//
// Measured (a matrix product of 8192^3 reaches 1183 TFLOP/s): 16384 tokens, 16
// heads of 128, 970 to 1030 us, 1.1 PFLOP/s, the matrix units 60% busy at the
// clock that the power limit leaves; 61 prompts of 9 to 467 tokens, 32 heads,
// 44 us, where 26 would move the bytes: half of a short workgroup's time is
// what comes before and after its tiles.
#include <type_traits>

#include "attention_device.h"

namespace fgs {

namespace {

using namespace attn;

constexpr int BN = 64;             // keys a tile
constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

struct FwdParams {
    const uint16_t *q, *k, *v;
    uint16_t* o;
    int64_t q_ld, q_hd, k_ld, k_hd, v_ld, v_hd, o_ld, o_hd;   // elements
    float* lse;
    const int32_t* cu;
    int64_t T;
    int S, hb_shift;     // 1 << hb_shift query heads a workgroup
    Order order;
    Divisor share;       // groups of heads that share a key head
    float scale;
};

// The wave's output rows again, for those (redo) that came out non-finite
// though what they see may be finite: the tile products below multiply a hidden
// key's zero probability with its value, and 0 * Inf is NaN.  The keys before
// the wave's rows, which all of these see, go by tiles as they did, with the m
// and l that the row has; the others, at most 32, one key at a time to the rows
// that see it.  So a row depends on the keys it sees and on nothing else, and
// the cost stays near that of the wave's first pass.  Nothing is done if no NaN
// or Inf is among the values of the wave's last tile, the only one with hidden
// keys.  A call, with the kernel's arguments by their address, so that the
// kernel's loop keeps its registers.  `lds`: 2 * 32 rows of D that are the wave's own.
typedef const __attribute__((address_space(4))) FwdParams* KernelArgs;
template <int D>
__device__ __attribute__((noinline)) void rows_again(KernelArgs p, int start, int len, int head, int kv_head, int w0,
                                                     float m, float l, bool redo, uint32_t lds)
{
    constexpr int TILE = 32 * D * 2;
    // the same in every lane, which a call does not tell the compiler
    start = __builtin_amdgcn_readfirstlane(start), len = __builtin_amdgcn_readfirstlane(len);
    head = __builtin_amdgcn_readfirstlane(head), kv_head = __builtin_amdgcn_readfirstlane(kv_head);
    w0 = __builtin_amdgcn_readfirstlane(w0), lds = __builtin_amdgcn_readfirstlane(lds);
    const int lane = threadIdx.x & 63, half = lane >> 5, last = len - 1, row = min(w0 + (lane & 31), last);
    const int64_t k_ld = p->k_ld, v_ld = p->v_ld, token = start + row;
    const uint16_t* k_seq = p->k + start * k_ld + kv_head * p->k_hd;
    const uint16_t* v_seq = p->v + start * v_ld + kv_head * p->v_hd;
    if (!rows_non_finite<D, BN>(v_seq, v_ld, w0, last, lane)) return;

    const uint16_t* q_row = p->q + token * p->q_ld + head * p->q_hd;
    bf16x8 q[D / 16];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) q[ks] = *reinterpret_cast<const bf16x8*>(q_row + 16 * ks + 8 * half);
    const float c = p->scale * LOG2E, mc = m * c;
    const uint32_t rows_at = lds + rows_address<D>(lane), tr_at = lds + tr_address<D>(lane);
    f32x16 o[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] = 0.0f;
#pragma unroll 1
    for (int k0 = 0; k0 < w0; k0 += 32) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");          // the last tile has been read
        stage<D, 32, 1>(uniform_ptr(k_seq + k0 * k_ld), (uint32_t)k_ld * 2, 31, lds, 0, lane);
        stage<D, 32, 1>(uniform_ptr(v_seq + k0 * v_ld), (uint32_t)v_ld * 2, 31, lds + TILE, 0, lane);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        f32x16 s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) s = mfma(read_rows_at(rows_at, ks, 0), q[ks], s);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -mc));
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
                o[dt] = mfma(read_tr_at<D>(tr_at, 16 * ks, dt, TILE), pack8(s, 8 * ks), o[dt]);
    }
#pragma unroll 1
    for (int key = w0; key < min(w0 + 32, len); ++key) {
        const float dot = dot_rows<D>(q_row, k_seq + key * k_ld, half);
        if (key <= row) add_row<D>(o, __builtin_amdgcn_exp2f(__builtin_fmaf(dot, c, -mc)), v_seq + key * v_ld, half);
    }
    store_row<D>(p->o + token * p->o_ld + head * p->o_hd, o, l == 0.0f ? 0.0f : 1.0f / l, lane, redo);
}

template <int D>
__global__ __launch_bounds__(256, 2) void attention_fwd_kernel(FwdParams p)
{
    constexpr int TILE = BN * D * 2;
    __shared__ __attribute__((aligned(256))) char lds[4 * TILE];   // K0 K1 V0 V1
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    const int rows = 128 >> p.hb_shift;
    const Mine mine = my_queries(p.cu, p.S, p.T, 7 - p.hb_shift, p.order, lane);
    const Where at = mine.at;
    const int group = mine.group;
    const int t0 = at.tile * rows;
    if (t0 >= at.len) return;
    const int head = (group << p.hb_shift) + (wave & ((1 << p.hb_shift) - 1));
    const int w0 = t0 + (wave >> p.hb_shift) * 32;          // the wave's first token in the segment
    const int row = w0 + (lane & 31);
    auto token_of = [&](int row) { return at.start + min(row, at.len - 1); };
    auto store = [&](const f32x16* o, float f, float lse) {
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));         // addresses formed here are not kept in registers until the end
        const int row = w0 + (lane & 31);
        const int64_t token = token_of(row);
        store_row<D>(p.o + token * p.o_ld + head * p.o_hd, o, f, lane, row < at.len);
        if (row < at.len && lane < 32) p.lse[head * p.T + token] = lse;
    };

    f32x16 o[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] = 0.0f;
    if (!at.sequence) return store(o, 0.0f, -__builtin_inff());       // tokens of no sequence see nothing

    const int kv_head = (int)divide(group, p.share);
    const uint16_t* q_row = p.q + token_of(row) * p.q_ld + head * p.q_hd;
    const uint16_t* k_seq = uniform_ptr(p.k + at.start * p.k_ld + kv_head * p.k_hd);
    const uint16_t* v_seq = uniform_ptr(p.v + at.start * p.v_ld + kv_head * p.v_hd);
    bf16x8 q[D / 16];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) q[ks] = *reinterpret_cast<const bf16x8*>(q_row + 16 * ks + 8 * half);

    const uint32_t base = lds_offset(lds);
    const int last = at.len - 1;
    const int n_tiles = (min(t0 + rows, at.len) + BN - 1) / BN;
    const int wave_keys = w0 < at.len ? min(w0 + 32, at.len) : 0;     // keys that some row of the wave sees
    const float c = p.scale * LOG2E;
    float m = 0.0f, l = 0.0f;                          // what the exponents are taken from; the lane half's sum
    const int wave_tiles = (wave_keys + BN - 1) / BN;

    auto load_k = [&](int n) {
        stage<D, BN, 4>(k_seq + (int64_t)n * BN * p.k_ld, (uint32_t)p.k_ld * 2, last - n * BN, base + (n & 1) * TILE,
                        wave, lane);
    };
    auto load_v = [&](int n) {
        stage<D, BN, 4>(v_seq + (int64_t)n * BN * p.v_ld, (uint32_t)p.v_ld * 2, last - n * BN,
                        base + (2 + (n & 1)) * TILE, wave, lane);
    };
    // The scores of a tile, and in between the exponents of `old` (with
    // exponents_too): one 16-deep step of both key halves, then the exponents
    // of as many registers, so that the vector unit works while the matrix
    // unit does; operands are read two steps ahead.  The compiler keeps
    // this order (the barriers to its scheduler), left to itself it reads
    // each operand right before its use.
    constexpr int KS = D / 16, CHUNK = 32 / KS;
    auto exponent_pair = [&](const f32x16 (&s)[2], int i, float mc, float (&sum)[2], uint32_t (&pr)[16]) {
        const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i / 16][i % 16], c, -mc));
        const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i / 16][i % 16 + 1], c, -mc));
        sum[0] += e0, sum[1] += e1;
        const bf16x2 w = {(__bf16)e0, (__bf16)e1};
        pr[i / 2] = __builtin_bit_cast(uint32_t, w);
    };
    auto scores = [&](auto exponents_too, int n, f32x16 (&s)[2], const f32x16 (&old)[2],
                      uint32_t (&pr)[16]) {
        const char* kt = lds + (n & 1) * TILE;
        const float mc = m * c;
        float sum[2] = {0.0f, 0.0f};
        bf16x8 k[KS][2];
        auto read = [&](int ks) {
#pragma unroll
            for (int t = 0; t < 2; ++t) k[ks][t] = read_rows<D>(kt, 32 * t, ks, lane);
        };
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
        read(0);
        read(1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks + 2 < KS) read(ks + 2);
#pragma unroll
            for (int t = 0; t < 2; ++t) s[t] = mfma(k[ks][t], q[ks], s[t]);
            if constexpr (decltype(exponents_too)::value)
#pragma unroll
                for (int i = ks * CHUNK; i < (ks + 1) * CHUNK; i += 2) {
                    exponent_pair(old, i, mc, sum, pr);
                    // here, and not together with the other branch's
                    asm volatile("" : "+v"(pr[i / 2]), "+v"(sum[0]), "+v"(sum[1]));
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        return sum[0] + sum[1];
    };
    auto row_top = [&](const f32x16 (&s)[2]) {
        float top = s[0][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, s[0][i]);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[1][i]);
        return fmaxf(top, swap_half(top));
    };
    auto hide = [&](int n, f32x16 (&s)[2]) {           // the diagonal: the keys after the row
        const int k0 = n * BN;
        if (k0 + BN <= w0) return;
        const int seen = min(row, last) - k0 - 4 * half;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (32 * t + acc_row(i, 0) > seen) s[t][i] = -__builtin_inff();
    };
    auto exponents = [&](const f32x16 (&s)[2], uint32_t (&pr)[16]) {
        float mc = m * c;
        asm volatile("" : "+v"(mc));                   // nothing of this is formed before a branch to here
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 32; i += 2) exponent_pair(s, i, mc, sum, pr);
        return sum[0] + sum[1];
    };
    // One tile: its exponents while the matrix unit forms the next tile's
    // scores, then its values' product.
    auto step = [&](int n, f32x16 (&s)[2], f32x16 (&next)[2]) {
        publish();
        if (n + 2 < n_tiles) load_k(n + 2);
        if (n + 1 < n_tiles) load_v(n + 1);
        if (n >= wave_tiles) return;
        hide(n, s);
        if (n == 0) {
            const float top = row_top(s);
            m = top == -__builtin_inff() ? 0.0f : top;
        }
        uint32_t pr[16];
        float sum;
        if (n + 1 < wave_tiles) sum = scores(std::true_type{}, n + 1, next, s, pr);
        else sum = exponents(s, pr);
        // m only has to keep exp2 in range: it moves when a row's exponents
        // pass 2^14, or when nothing of the row is above 2^-60 yet, so most
        // tiles never look for their maximum nor touch the output sums.  It
        // moves for those rows alone, or a row's bits would depend on others'.
        const bool moves = !(sum <= 16384.0f) || (l == 0.0f && sum < 0x1p-60f);
        if (__any(moves)) {
            const float top = row_top(s);
            const float here = moves ? 1.0f : 0.0f, other = swap_half(here), l_other = swap_half(l);
            const bool none = l + l_other == 0.0f, stays = here + other == 0.0f;
            const float to = stays ? m : none ? (top == -__builtin_inff() ? m : top) : fmaxf(m, top);
            const float old = none ? 1.0f : __builtin_amdgcn_exp2f((m - to) * c);
            m = to;
            l *= old;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[dt][i] *= old;
            sum = exponents(s, pr);
        }
        l += sum;
        // operands are read three products ahead, as above
        constexpr int F = 4 * (D / 32);
        const char* vt = lds + (2 + (n & 1)) * TILE;
        bf16x8 v[F];
        auto read = [&](int f) { v[f] = read_tr<D>(vt, 16 * (f / (D / 32)), f % (D / 32), lane); };
        read(0);
        read(1);
        read(2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < F; ++f) {
            if (f + 3 < F) read(f + 3);
            const int w = f / (D / 32) * 4;
            const u32x4 b = {pr[w], pr[w + 1], pr[w + 2], pr[w + 3]};
            o[f % (D / 32)] = mfma(v[f], __builtin_bit_cast(bf16x8, b), o[f % (D / 32)]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    load_k(0);
    load_v(0);
    if (n_tiles > 1) load_k(1);
    registers_landed();
    publish();
    f32x16 sa[2], sb[2];
    uint32_t unused[16];
    if (wave_tiles > 0) scores(std::false_type{}, 0, sa, sb, unused);
    for (int n = 0; n < n_tiles; n += 2) {
        step(n, sa, sb);
        if (n + 1 < n_tiles) step(n + 1, sb, sa);
    }
    publish();                                 // from here on each wave has a part of the tiles' place to itself
    if (w0 >= at.len) return;
    l += swap_half(l);
    const bool redo = row < at.len && non_finite<D>(o);
    store(o, l == 0.0f ? 0.0f : 1.0f / l, m * p.scale + __logf(l));
    static_assert(2 * 32 * D * 2 <= TILE, "two tiles of 32 rows");
    if (__any(redo))
        rows_again<D>((KernelArgs)__builtin_amdgcn_kernarg_segment_ptr(), (int)at.start, at.len, head, kv_head, w0, m, l,
                      redo, base + wave * TILE);
}

} // namespace

hipError_t launch_attention_fwd(const AttentionArgs& a, hipStream_t stream)
{
    FwdParams p{};
    p.q = (const uint16_t*)a.q.data, p.k = (const uint16_t*)a.k.data, p.v = (const uint16_t*)a.v.data;
    p.o = (uint16_t*)a.out.data;
    p.q_ld = a.q.ld_token, p.q_hd = a.q.ld_head, p.k_ld = a.k.ld_token, p.k_hd = a.k.ld_head;
    p.v_ld = a.v.ld_token, p.v_hd = a.v.ld_head, p.o_ld = a.out.ld_token, p.o_hd = a.out.ld_head;
    p.lse = a.lse, p.cu = a.cu_seqlens, p.T = a.T, p.S = a.S;
    const int shared = a.H / a.Hk;
    p.hb_shift = shared % 4 == 0 ? 2 : shared % 2 == 0 ? 1 : 0;
    p.order = Order((int)(a.T / (128 >> p.hb_shift)) + a.S + 2, a.H >> p.hb_shift);
    p.share = Divisor((uint32_t)(shared >> p.hb_shift));
    p.scale = a.scale;
    const dim3 grid((unsigned)((int64_t)p.order.tiles * p.order.groups));
    if (a.D == 128)
        attention_fwd_kernel<128><<<grid, 256, 0, stream>>>(p);
    else
        attention_fwd_kernel<64><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
}

} // namespace fgs
