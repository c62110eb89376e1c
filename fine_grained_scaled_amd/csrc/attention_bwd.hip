// attention_bwd.hip -- the gradients of causal attention over packed
// sequences with grouped heads, on gfx950.
//
// With p = exp(z - lse) the forward pass's probabilities and
// delta[t] = sum_d dout[t][d] out[t][d]:
//   dv[u] = sum_t p[t][u] dout[t]
//   ds[t][u] = p[t][u] (dout[t] . v[u] - delta[t])
//   dq[t] = scale sum_u ds[t][u] k[u],  dk[u] = scale sum_t ds[t][u] q[t],
// t over the tokens that see u and, for dk and dv, over the query heads that
// share the key head.  p and ds are recomputed in FP32 and rounded to BF16
// once for the products; all sums are FP32.
//
// A row's p is about 1 / (its keys), so the first rows of a sequence weigh
// most in every gradient, and there dout . v - delta cancels: row 0 has
// ds = 0.  The rows that see one tile of keys (the first 64) therefore take
// delta from their own p and dout . v instead of the rounded out, and they
// (for dk and dv the first 32) hand p and ds to the products as two BF16
// terms, value and remainder.  That is one more set of products in one tile of
// a sequence, and it takes the error of dq, dk and dv against 64 bits from 1.5
// to 1.3 times that of the results' own rounding.
//
// Two kernels, each with its sums in registers: one owns query rows (dq, and
// delta), the other owns keys (dk, dv) and walks the query heads of their
// group.  They compute the scores twice, 14 D operations a pair instead of
// 10, and in return no sum crosses workgroups: no atomics, no FP32 copy of
// dq, and the same bits on every run.
//
// Measured: 8192 tokens, 32 heads of 128 over 8 key heads, dq 700 to 775 us and
// dk, dv 1020 to 1120 us, 1.0 to 1.1 PFLOP/s of executed products, near the rate
// of a large matrix product (1183 TFLOP/s); 7 documents in the same tokens,
// 254 and 352 us; 9 documents in 4099 tokens, 16 heads of 64, 31 and 36 us.
#include <algorithm>
#include <type_traits>

#include "attention_device.h"

namespace fgs {

namespace {

using namespace attn;

constexpr float LOG2E = 1.44269504088896340736f;

struct BwdParams {
    const uint16_t *q, *k, *v, *o, *dout;
    uint16_t *dq, *dk, *dv;
    int64_t q_ld, q_hd, k_ld, k_hd, v_ld, v_hd, o_ld, o_hd, do_ld, do_hd;   // elements
    int64_t dq_ld, dq_hd, dk_ld, dk_hd, dv_ld, dv_hd;
    const float* lse;
    float* ws;            // [H][T] -lse / scale, then [H][T] -delta
    const int32_t* cu;
    int64_t T;
    int S, H, hb_shift, group_heads;
    Order order, kv_order;
    Divisor share;
    Split split;
    float* shares;        // split key tiles: [slot][dk, dv][4 waves][32 keys x D]
    int* arrived;         // [slot]: the parts that are done, at the tile's first slot
    int slots, kv_slots;  // of all heads, of one
    float scale;
};

constexpr int BN = 64;    // keys a tile of the dq kernel
constexpr int QN = 64;    // query rows a tile of the dk, dv kernel
constexpr int KN = 128;   // keys a workgroup of it (1 << 7)
constexpr int FIRST = 64; // rows at the start of a sequence that are kept more exactly,
constexpr int REST = 32;  // and those whose remainders go into dk and dv
static_assert(FIRST == BN && KN <= 2 * BN && REST == 32, "one tile of keys, 32 queries");

// What pack8() drops, rounded in turn.
__device__ __forceinline__ bf16x8 pack8_rest(const f32x16& s, int i0)
{
    bf16x8 r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = (__bf16)(s[i0 + j] - (float)(__bf16)s[i0 + j]);
    return r;
}

// The wave's rows of dq again, for those (redo) that came out non-finite though
// what they see may be finite: the tile products multiply a hidden pair's zero
// with a row of the tile, and 0 * Inf is NaN.  The keys before the wave's rows,
// which all of these see, go by tiles as they did, the others, at most 32, one
// pair at a time and every hidden pair left out, so the cost stays near that of
// the wave's first pass.  Nothing is done if no NaN or Inf is among the keys of
// the tiles with hidden pairs.  A call, with the kernel's arguments by their
// address, so that the kernel's loops keep their registers.
// `lds`: 2 * 32 rows of D that are the wave's own.
typedef const __attribute__((address_space(4))) BwdParams* KernelArgs;
template <int D>
__device__ __attribute__((noinline)) void dq_again(KernelArgs p, int start, int len, int head, int kv_head, int w0,
                                                   float from, float delta, bool redo, uint32_t lds)
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
    if (!rows_non_finite<D, BN>(k_seq, k_ld, w0, last, lane)) return;

    const uint16_t* q_row = p->q + token * p->q_ld + head * p->q_hd;
    const uint16_t* do_row = p->dout + token * p->do_ld + head * p->do_hd;
    const float c = p->scale * LOG2E;
    const uint32_t rows_at = lds + rows_address<D>(lane), tr_at = lds + tr_address<D>(lane);
    f32x16 dq[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[dt][i] = 0.0f;
#pragma unroll 1
    for (int k0 = 0; k0 < w0; k0 += 32) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");          // the last tile has been read
        stage<D, 32, 1>(uniform_ptr(k_seq + k0 * k_ld), (uint32_t)k_ld * 2, 31, lds, 0, lane);
        stage<D, 32, 1>(uniform_ptr(v_seq + k0 * v_ld), (uint32_t)v_ld * 2, 31, lds + TILE, 0, lane);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        f32x16 s, dp;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = from, dp[i] = delta;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            s = mfma(read_rows_at(rows_at, ks, 0), *reinterpret_cast<const bf16x8*>(q_row + 16 * ks + 8 * half), s);
            dp = mfma(read_rows_at(rows_at, ks, TILE), *reinterpret_cast<const bf16x8*>(do_row + 16 * ks + 8 * half), dp);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(s[i] * c) * dp[i];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
                dq[dt] = mfma(read_tr_at<D>(tr_at, 16 * ks, dt, 0), pack8(s, 8 * ks), dq[dt]);
    }
#pragma unroll 1
    for (int key = w0; key < min(w0 + 32, len); ++key) {
        const uint16_t* k = k_seq + key * k_ld;
        const float z = dot_rows<D>(q_row, k, half), dp = dot_rows<D>(do_row, v_seq + key * v_ld, half);
        if (key <= row) add_row<D>(dq, __builtin_amdgcn_exp2f((z + from) * c) * (dp + delta), k, half);
    }
    store_row<D>(p->dq + token * p->dq_ld + head * p->dq_hd, dq, p->scale, lane, redo);
}

// The wave's keys of dk and dv again, for those (redo) that came out non-finite
// though what they see may be finite: the wave's first 32 queries of each head,
// where pairs are hidden, one pair at a time, all later ones by tiles, which are
// right as they are.  Nothing is done if no NaN or Inf is among those first
// queries.  A call, with the kernel's arguments by their address: inlined, this
// path cost the kernel's loops 7% by what the compiler kept in registers for it.
// `lds`: 2 * 32 rows of D that are the wave's own.
template <int D>
__device__ __attribute__((noinline)) void dkv_again(KernelArgs p, int start, int len, int kv_head, int w0, bool redo,
                                                    uint32_t lds)
{
    constexpr int TILE = 32 * D * 2;
    start = __builtin_amdgcn_readfirstlane(start), len = __builtin_amdgcn_readfirstlane(len);
    kv_head = __builtin_amdgcn_readfirstlane(kv_head);
    w0 = __builtin_amdgcn_readfirstlane(w0), lds = __builtin_amdgcn_readfirstlane(lds);
    const int lane = threadIdx.x & 63, half = lane >> 5, key = w0 + (lane & 31), last = len - 1;
    const int first_head = kv_head * p->group_heads, heads_end = first_head + p->group_heads;
    const int64_t q_ld = p->q_ld, do_ld = p->do_ld;
    bool hidden = false;
#pragma unroll 1
    for (int h = first_head; h < heads_end; ++h)
        hidden |= rows_non_finite<D, 32>(p->q + start * q_ld + h * p->q_hd, q_ld, w0, last, lane) ||
                  rows_non_finite<D, 32>(p->dout + start * do_ld + h * p->do_hd, do_ld, w0, last, lane);
    if (!hidden) return;

    const float c = p->scale * LOG2E;
    const int64_t own = (int64_t)start + min(key, last);
    const uint16_t* k_row = p->k + own * p->k_ld + kv_head * p->k_hd;
    const uint16_t* v_row = p->v + own * p->v_ld + kv_head * p->v_hd;
    const uint32_t rows_at = lds + rows_address<D>(lane), tr_at = lds + tr_address<D>(lane);
    f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[dt][i] = dv[dt][i] = 0.0f;
#pragma unroll 1
    for (int h = first_head; h < heads_end; ++h) {
        const float* from = p->ws + (int64_t)h * p->T + start;
        const float* delta = p->ws + (int64_t)(p->H + h) * p->T + start;
        const uint16_t* q_seq = p->q + start * q_ld + h * p->q_hd;
        const uint16_t* g_seq = p->dout + start * do_ld + h * p->do_hd;
#pragma unroll 1
        for (int t = w0; t < min(w0 + 32, len); ++t) {
            const uint16_t *q = q_seq + t * q_ld, *g = g_seq + t * do_ld;
            const float z = dot_rows<D>(q, k_row, half), dp = dot_rows<D>(g, v_row, half);
            if (t < key) continue;
            const float pr = __builtin_amdgcn_exp2f((z + from[t]) * c);
            add_row<D>(dv, pr, g, half);
            add_row<D>(dk, pr * (dp + delta[t]), q, half);
        }
#pragma unroll 1
        for (int q0 = w0 + 32; q0 < len; q0 += 32) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the last tile has been read
            stage<D, 32, 1>(uniform_ptr(q_seq + q0 * q_ld), (uint32_t)q_ld * 2, last - q0, lds, 0, lane);
            stage<D, 32, 1>(uniform_ptr(g_seq + q0 * do_ld), (uint32_t)do_ld * 2, last - q0, lds + TILE, 0, lane);
            f32x16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int t = min(q0 + acc_row(i, half), last);
                s[i] = from[t], dp[i] = delta[t];
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                s = mfma(read_rows_at(rows_at, ks, 0), *reinterpret_cast<const bf16x8*>(k_row + 16 * ks + 8 * half), s);
                dp = mfma(read_rows_at(rows_at, ks, TILE), *reinterpret_cast<const bf16x8*>(v_row + 16 * ks + 8 * half),
                          dp);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[i] = q0 + acc_row(i, half) > last ? 0.0f : __builtin_amdgcn_exp2f(s[i] * c);
                dp[i] = q0 + acc_row(i, half) > last ? 0.0f : dp[i] * s[i];
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const bf16x8 pr = pack8(s, 8 * ks), ds = pack8(dp, 8 * ks);
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt) {
                    dv[dt] = mfma(read_tr_at<D>(tr_at, 16 * ks, dt, TILE), pr, dv[dt]);
                    dk[dt] = mfma(read_tr_at<D>(tr_at, 16 * ks, dt, 0), ds, dk[dt]);
                }
            }
        }
    }
    store_row<D>(p->dk + own * p->dk_ld + kv_head * p->dk_hd, dk, p->scale, lane, redo);
    store_row<D>(p->dv + own * p->dv_ld + kv_head * p->dv_hd, dv, 1.0f, lane, redo);
}

// dq: 4 waves as in the forward kernel (HB heads x 128 / HB tokens, 32 rows a
// wave), S^T = K Q^T and dP^T = V dO^T a 32-key step, dQ^T += K^T dS^T.
template <int D>
__global__ __launch_bounds__(256, D == 64 ? 3 : 2) void attention_dq_kernel(BwdParams p)
{
    constexpr int TILE = BN * D * 2;
    __shared__ __attribute__((aligned(256))) char lds[4 * TILE];   // K0 K1 V0 V1
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.slots; i += blockDim.x) p.arrived[i] = 0;
    const int rows = 128 >> p.hb_shift;
    const Mine mine = my_queries(p.cu, p.S, p.T, 7 - p.hb_shift, p.order, lane);
    const Where at = mine.at;
    const int group = mine.group;
    const int t0 = at.tile * rows;
    if (t0 >= at.len) return;
    const int head = (group << p.hb_shift) + (wave & ((1 << p.hb_shift) - 1));
    const int w0 = t0 + (wave >> p.hb_shift) * 32;
    const int row = w0 + (lane & 31);
    const bool write = row < at.len;
    const int64_t token = at.start + (write ? row : at.len - 1);
    uint16_t* dq_row = p.dq + token * p.dq_ld + head * p.dq_hd;

    f32x16 dq[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[dt][i] = 0.0f;
    if (!at.sequence) {
        store_row<D>(dq_row, dq, 0.0f, lane, write);
        return;
    }
    const int kv_head = (int)divide(group, p.share);
    const uint16_t* q_row = p.q + token * p.q_ld + head * p.q_hd;
    const uint16_t* do_row = p.dout + token * p.do_ld + head * p.do_hd;
    const uint16_t* o_row = p.o + token * p.o_ld + head * p.o_hd;
    const uint16_t* k_seq = uniform_ptr(p.k + at.start * p.k_ld + kv_head * p.k_hd);
    const uint16_t* v_seq = uniform_ptr(p.v + at.start * p.v_ld + kv_head * p.v_hd);
    bf16x8 q[D / 16], g[D / 16];
    float delta = 0.0f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        q[ks] = *reinterpret_cast<const bf16x8*>(q_row + 16 * ks + 8 * half);
        g[ks] = *reinterpret_cast<const bf16x8*>(do_row + 16 * ks + 8 * half);
        const bf16x8 o = *reinterpret_cast<const bf16x8*>(o_row + 16 * ks + 8 * half);
#pragma unroll
        for (int j = 0; j < 8; ++j) delta = __builtin_fmaf((float)g[ks][j], (float)o[j], delta);
    }
    delta += swap_half(delta);
    // the scores start from -lse / scale, so that p = exp2(c s); a row whose
    // scores are all -Inf has p = 0
    const float lse = p.lse[head * p.T + token];
    const float from = lse == -__builtin_inff() ? 0.0f : -lse / p.scale;
    delta = -delta;

    const uint32_t base = lds_offset(lds);
    const int last = at.len - 1;
    const int n_tiles = (min(t0 + rows, at.len) + BN - 1) / BN;
    const int wave_keys = w0 >= FIRST && w0 < at.len ? min(w0 + 32, at.len) : 0;   // the first rows come after the loop
    const float c = p.scale * LOG2E;
    auto load = [&](int n, int buf) {
        const int k0 = n * BN;
        stage<D, BN, 4>(k_seq + (int64_t)k0 * p.k_ld, (uint32_t)p.k_ld * 2, last - k0, base + buf * TILE, wave, lane);
        stage<D, BN, 4>(v_seq + (int64_t)k0 * p.v_ld, (uint32_t)p.v_ld * 2, last - k0, base + (2 + buf) * TILE, wave,
                        lane);
    };
    load(0, 0);
    registers_landed();
    for (int n = 0; n < n_tiles; ++n) {
        const int buf = n & 1;
        publish();
        if (n + 1 < n_tiles) load(n + 1, buf ^ 1);
        const char* kt = lds + buf * TILE;
        const char* vt = lds + (2 + buf) * TILE;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int k0 = n * BN + 32 * t;
            if (k0 >= wave_keys) continue;
            f32x16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = from, dp[i] = delta;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                s = mfma(read_rows<D>(kt, 32 * t, ks, lane), q[ks], s);
                dp = mfma(read_rows<D>(vt, 32 * t, ks, lane), g[ks], dp);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(s[i] * c) * dp[i];
            if (k0 + 31 > w0) {
                const int seen = min(row, last) - k0 - 4 * half;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (acc_row(i, 0) > seen) s[i] = 0.0f;
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const bf16x8 ds = pack8(s, 8 * ks);
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt)
                    dq[dt] = mfma(read_tr<D>(kt, 32 * t + 16 * ks, dt, lane), ds, dq[dt]);
            }
        }
    }
    if (w0 < FIRST && w0 < at.len) {                   // their tile is still in LDS
        f32x16 s[2], dp[2];
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] = from, dp[t][i] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                s[t] = mfma(read_rows<D>(lds, 32 * t, ks, lane), q[ks], s[t]);
                dp[t] = mfma(read_rows<D>(lds + 2 * TILE, 32 * t, ks, lane), g[ks], dp[t]);
            }
            const int seen = min(row, last) - 32 * t - 4 * half;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[t][i] = acc_row(i, 0) > seen ? 0.0f : __builtin_amdgcn_exp2f(s[t][i] * c);
                dp[t][i] = acc_row(i, 0) > seen ? 0.0f : dp[t][i];
                sum = __builtin_fmaf(s[t][i], dp[t][i], sum);
            }
        }
        delta = -(sum + swap_half(sum));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] *= dp[t][i] + delta;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const bf16x8 ds = pack8(s[t], 8 * ks), rest = pack8_rest(s[t], 8 * ks);
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt) {
                    const bf16x8 x = read_tr<D>(lds, 32 * t + 16 * ks, dt, lane);
                    dq[dt] = mfma(x, ds, mfma(x, rest, dq[dt]));
                }
            }
        }
    }
    publish();                                 // from here on each wave has a part of the tiles' place to itself
    if (w0 >= at.len) return;
    if (write && half == 0) {
        p.ws[head * p.T + token] = from;
        p.ws[(p.H + head) * p.T + token] = delta;
    }
    const bool redo = write && non_finite<D>(dq);
    store_row<D>(dq_row, dq, p.scale, lane, write);
    static_assert(2 * 32 * D * 2 <= TILE, "two tiles of 32 rows");
    if (__any(redo))
        dq_again<D>((KernelArgs)__builtin_amdgcn_kernarg_segment_ptr(), (int)at.start, at.len, head, kv_head, w0, from,
                    delta, redo, base + wave * TILE);
}

// dk and dv: 8 waves, two sets of 4 that own the same 4 x 32 keys, whose key
// and value rows stay in registers.  Tiles of 64 query rows and their
// gradients pass through LDS, head after head of the group, the sets taking
// turns; at the end the second set hands its sums to the first through LDS.
// So a workgroup fills a compute unit with two waves a SIMD and the longest
// of them takes half as long.  S = Q K^T and dP = dO V^T leave a lane one key
// and 16 queries a step, again the B operands of dV^T += dO^T P and
// dK^T += Q^T dS; both start from the row's value (-lse / scale, -delta)
// instead of zero.  With 64-wide heads a third of a SIMD's registers is a wave's
// limit, dkv_again() included, so that the next workgroup starts when one of
// this one's sets is done (4099 tokens: 38.0 us with 249 registers, 35.6 so).
template <int D>
__global__ __launch_bounds__(512, D == 64 ? 3 : 2) void attention_dkv_kernel(BwdParams p)
{
    constexpr int TILE = QN * D * 2;
    constexpr int STAGE = 2 * TILE + 2 * 64 * 4;          // Q, dO, then the row values, 64 a copy
    __shared__ __attribute__((aligned(256))) char lds_all[4 * STAGE];
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int set = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
    char* lds = lds_all + set * 2 * STAGE;
    const Mine mine = my_keys(p.cu, p.S, p.T, 7, p.kv_order, p.split, lane);
    const Where at = mine.at;
    const int kv_head = mine.group;
    const int k0 = at.tile * KN;
    if (k0 >= at.len) return;
    const int w0 = k0 + wave * 32;
    const int key = w0 + (lane & 31);
    const bool write = key < at.len && set == 0;
    auto token_of = [&](int key) { return at.start + min(key, at.len - 1); };

    f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[dt][i] = dv[dt][i] = 0.0f;
    auto store = [&](bool write) {
        int key_now = key;                     // addresses formed here are not kept in registers until the end
        asm volatile("" : "+v"(key_now));
        const int64_t token = token_of(key_now);
        store_row<D>(p.dk + token * p.dk_ld + kv_head * p.dk_hd, dk, p.scale, lane, write);
        store_row<D>(p.dv + token * p.dv_ld + kv_head * p.dv_hd, dv, 1.0f, lane, write);
    };
    if (!at.sequence) return store(write);
    const int64_t token = token_of(key);
    const uint16_t* k_row = p.k + token * p.k_ld + kv_head * p.k_hd;
    const uint16_t* v_row = p.v + token * p.v_ld + kv_head * p.v_hd;
    bf16x8 k[D / 16], v[D / 16];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        k[ks] = *reinterpret_cast<const bf16x8*>(k_row + 16 * ks + 8 * half);
        v[ks] = *reinterpret_cast<const bf16x8*>(v_row + 16 * ks + 8 * half);
    }
    const uint32_t base = lds_offset(lds);
    const int last = at.len - 1;
    const int q_first = k0 / QN, q_tiles = (at.len + QN - 1) / QN - q_first;
    // this part's steps: heads of the group and query tiles within them
    const int all_tiles = q_tiles * p.group_heads;
    int begin = 0, steps = all_tiles;
    if (at.parts > 1) {
        begin = (int)((int64_t)all_tiles * at.part / at.parts);
        steps = (int)((int64_t)all_tiles * (at.part + 1) / at.parts) - begin;
    }
    const float c = p.scale * LOG2E;
    // the head and the query tile of the set's step
    int head = kv_head * p.group_heads + begin / q_tiles, q_index = begin % q_tiles + set;
    auto forward = [&](int& h, int& i) {
        while (i >= q_tiles) i -= q_tiles, ++h;
    };
    forward(head, q_index);
    auto load = [&](int head, int q_index, int stage_at) {
        const int q0 = (q_first + q_index) * QN;
        const uint16_t* q = uniform_ptr(p.q + (at.start + q0) * p.q_ld + head * p.q_hd);
        const uint16_t* g = uniform_ptr(p.dout + (at.start + q0) * p.do_ld + head * p.do_hd);
        const uint32_t to = base + stage_at * STAGE;
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));         // nothing of the copies' addresses stays in registers between them
        stage<D, QN, 4>(q, (uint32_t)p.q_ld * 2, last - q0, to, wave, lane);
        stage<D, QN, 4>(g, (uint32_t)p.do_ld * 2, last - q0, to + TILE, wave, lane);
        if (wave < 2)
            g2lds4(uniform_ptr(p.ws + ((int64_t)wave * p.H + head) * p.T + at.start + q0),
                   4 * min(lane & (QN - 1), last - q0), to + 2 * TILE + wave * 256);
    };
    // 32 queries and the wave's 32 keys, with p and ds or with what their
    // rounding leaves.  256 registers hold the sums, the
    // keys and values and two score tiles with little to spare: operands are
    // read two products ahead, which the scheduler barriers keep in place.
    const uint32_t rows_at = rows_address<D>(lane), tr_at = tr_address<D>(lane);
    auto step = [&](auto rest, uint32_t tile, const float* row_value, int q0) {
        f32x16 s, dp;
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(row_value + 2 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i + j] = a[j];
        }
        constexpr int KS = D / 16;
        bf16x8 x[2 * KS];
        uint32_t at_row = tile + rows_at;
        asm volatile("" : "+v"(at_row));
        auto read = [&](int f) { x[f] = read_rows_at(at_row, f % KS, f < KS ? 0 : TILE); };
        read(0);
        read(1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < 2 * KS; ++f) {
            if (f + 2 < 2 * KS) read(f + 2);
            if (f == KS - 4)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const f32x4 d = *reinterpret_cast<const f32x4*>(row_value + 64 + 2 * i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) dp[i + j] = d[j];
                }
            if (f < KS) s = mfma(x[f], k[f], s);
            else dp = mfma(x[f], v[f - KS], dp);
            __builtin_amdgcn_sched_barrier(0);
        }
        constexpr int DT = D / 32, F = 4 * DT;
        bf16x8 y[F];
        uint32_t at_tr = tile + tr_at;
        asm volatile("" : "+v"(at_tr));
        auto read2 = [&](int f) {       // of dv, then of dk: rows 16 (f / DT % 2), columns 32 (f % DT)
            y[f] = read_tr_at<D>(at_tr, 16 * (f / DT % 2), f % DT, f < 2 * DT ? TILE : 0);
        };
        read2(0);
        read2(1);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = __builtin_amdgcn_exp2f(s[i] * c);
            dp[i] *= s[i];
        }
        if (q0 < w0 + 31 || q0 + 32 > at.len) {
            int lane = threadIdx.x & 63;
            asm volatile("" : "+v"(lane));     // the key's number is not kept in a register for this
            const int first = 4 * (lane >> 5), from = w0 + (lane & 31) - q0 - first, to = at.len - q0 - first;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (acc_row(i, 0) < from || acc_row(i, 0) >= to) s[i] = dp[i] = 0.0f;
        }
        if constexpr (decltype(rest)::value) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] -= (float)(__bf16)s[i], dp[i] -= (float)(__bf16)dp[i];
        }
        bf16x8 pr[2], ds[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) pr[ks] = pack8(s, 8 * ks), ds[ks] = pack8(dp, 8 * ks);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < F; ++f) {
            if (f + 2 < F) read2(f + 2);
            if (f < 2 * DT) dv[f % DT] = mfma(y[f], pr[f / DT], dv[f % DT]);
            else dk[f % DT] = mfma(y[f], ds[f / DT - 2], dk[f % DT]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const int set_steps = (steps + 1 - set) / 2, all_steps = (steps + 1) / 2;
    if (set_steps > 0) load(head, q_index, 0);
    registers_landed();
    // The first key tile of a sequence adds the first rows' remainders, in a
    // loop of its own: the choice alone cost the other one 10%.
    auto walk = [&](auto first_tile) {
        for (int m = 0; m < all_steps; ++m) {
            publish();
            const int q0 = (q_first + q_index) * QN;
            q_index += 2;
            forward(head, q_index);
            if (m + 1 < set_steps) load(head, q_index, (m + 1) & 1);
            if (m >= set_steps) continue;
            const uint32_t tile = base + (m & 1) * STAGE;
            const float* row_value = reinterpret_cast<const float*>(lds + (m & 1) * STAGE + 2 * TILE) + 4 * half;
            if constexpr (decltype(first_tile)::value)
                if (q0 < REST && w0 < REST) step(std::true_type{}, tile, row_value, q0);
#pragma unroll
            for (int t = 0; t < QN / 32; ++t)
                if (q0 + 32 * t + 31 >= w0 && q0 + 32 * t < at.len)
                    step(std::false_type{}, tile + 32 * t * (D * 2), row_value + 32 * t, q0 + 32 * t);
        }
    };
    if (k0 < REST) walk(std::true_type{});
    else walk(std::false_type{});
    // the second set's sums, 32 keys x D of FP32 a wave, dk and then dv
    static_assert(4 * 32 * D * 4 <= 4 * STAGE, "the exchange fits");
    f32x4* swap = reinterpret_cast<f32x4*>(lds_all) + wave * (32 * D / 4) + lane;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        f32x16* acc = pass ? dv : dk;
        publish();
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (set)
                    swap[64 * (4 * dt + g)] = f32x4{acc[dt][4 * g], acc[dt][4 * g + 1], acc[dt][4 * g + 2],
                                                    acc[dt][4 * g + 3]};
        publish();
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (!set) {
                    const f32x4 o = swap[64 * (4 * dt + g)];
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[dt][4 * g + j] += o[j];
                }
    }
    if (at.parts > 1) {
        // The parts' sums meet in memory: each writes its own, the last one to
        // arrive adds them in the parts' order, so the bits do not depend on
        // which one that is.  Nothing waits for another workgroup.  Stores and
        // loads go past the L2 of their XCD one by one; a fence instead would
        // write all of it back (2048 tokens, 16 heads of 64: +40 us).
        constexpr int PER_WAVE = 32 * D / 2, PER_SLOT = 2 * 4 * PER_WAVE;      // in pairs
        const int first = kv_head * p.kv_slots + at.slot - at.part;
        uint64_t* mine = reinterpret_cast<uint64_t*>(p.shares) + (int64_t)(first + at.part) * PER_SLOT +
                         wave * PER_WAVE + lane;
        if (!set)
#pragma unroll
            for (int pass = 0; pass < 2; ++pass)
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        const f32x16& acc = pass ? dv[dt] : dk[dt];
                        const uint64_t x = (uint64_t)as_u32(acc[2 * g + 1]) << 32 | as_u32(acc[2 * g]);
                        __hip_atomic_store(mine + pass * 4 * PER_WAVE + 64 * (8 * dt + g), x, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
                    }
        publish();                             // every wave's stores are done
        int* ticket = reinterpret_cast<int*>(lds_all);
        if (threadIdx.x == 0)
            *ticket = __hip_atomic_fetch_add(p.arrived + first, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        publish();
        if (set || *ticket != at.parts - 1) return;
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) dk[dt][i] = dv[dt][i] = 0.0f;
        const uint64_t* from = mine - (int64_t)at.part * PER_SLOT;
#pragma unroll 1
        for (int part = 0; part < at.parts; ++part, from += PER_SLOT)
#pragma unroll
            for (int pass = 0; pass < 2; ++pass)
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        const uint64_t x = __hip_atomic_load(from + pass * 4 * PER_WAVE + 64 * (8 * dt + g),
                                                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                        f32x16& acc = pass ? dv[dt] : dk[dt];
                        acc[2 * g] += as_f32((uint32_t)x);
                        acc[2 * g + 1] += as_f32((uint32_t)(x >> 32));
                    }
    }
    if (set) return;
    publish();                                 // from here on each wave left has a part of the tiles' place to itself
    if (w0 >= at.len) return;
    const bool bad = non_finite<D>(dk), redo = write && (non_finite<D>(dv) || bad);
    store(write);
    static_assert(2 * 32 * D * 2 <= STAGE && STAGE % 256 == 0, "two tiles of 32 rows");
    if (__any(redo))
        dkv_again<D>((KernelArgs)__builtin_amdgcn_kernarg_segment_ptr(), (int)at.start, at.len, kv_head, w0, redo,
                     lds_offset(lds_all) + wave * STAGE);
}

} // namespace

hipError_t launch_attention_bwd(const AttentionArgs& a, hipStream_t stream)
{
    BwdParams p{};
    p.q = (const uint16_t*)a.q.data, p.k = (const uint16_t*)a.k.data, p.v = (const uint16_t*)a.v.data;
    p.o = (const uint16_t*)a.out.data, p.dout = (const uint16_t*)a.dout.data;
    p.dq = (uint16_t*)a.dq.data, p.dk = (uint16_t*)a.dk.data, p.dv = (uint16_t*)a.dv.data;
    p.q_ld = a.q.ld_token, p.q_hd = a.q.ld_head, p.k_ld = a.k.ld_token, p.k_hd = a.k.ld_head;
    p.v_ld = a.v.ld_token, p.v_hd = a.v.ld_head, p.o_ld = a.out.ld_token, p.o_hd = a.out.ld_head;
    p.do_ld = a.dout.ld_token, p.do_hd = a.dout.ld_head, p.dq_ld = a.dq.ld_token, p.dq_hd = a.dq.ld_head;
    p.dk_ld = a.dk.ld_token, p.dk_hd = a.dk.ld_head, p.dv_ld = a.dv.ld_token, p.dv_hd = a.dv.ld_head;
    p.lse = a.lse, p.ws = a.delta, p.cu = a.cu_seqlens, p.T = a.T, p.S = a.S, p.H = a.H;
    const int shared = a.H / a.Hk;
    p.hb_shift = shared % 4 == 0 ? 2 : shared % 2 == 0 ? 1 : 0;
    p.group_heads = shared;
    p.order = Order((int)(a.T / (128 >> p.hb_shift)) + a.S + 2, a.H >> p.hb_shift);
    p.share = Divisor((uint32_t)(shared >> p.hb_shift));
    p.scale = a.scale;
    const dim3 grid((unsigned)((int64_t)p.order.tiles * p.order.groups));
    // at most `extra` workgroups a head beyond one a tile, so at most 2 extra
    // of split tiles (each has two at least)
    p.split.extra = a.T >= ATTENTION_SPLIT_TOKENS ? ATTENTION_SLOTS / 2 / a.Hk : 0;
    p.split.least = std::max(1, 8 / shared);
    p.split.fair = (float)a.Hk / (float)device_cus();
    p.kv_slots = 2 * p.split.extra;
    p.slots = p.kv_slots * a.Hk;
    p.shares = a.shares, p.arrived = a.arrived;
    p.kv_order = Order((int)(a.T / KN) + a.S + 2 + p.split.extra, a.Hk);
    const dim3 grid_kv((unsigned)((int64_t)p.kv_order.tiles * a.Hk));
    if (a.D == 128) {
        attention_dq_kernel<128><<<grid, 256, 0, stream>>>(p);
        attention_dkv_kernel<128><<<grid_kv, 512, 0, stream>>>(p);
    } else {
        attention_dq_kernel<64><<<grid, 256, 0, stream>>>(p);
        attention_dkv_kernel<64><<<grid_kv, 512, 0, stream>>>(p);
    }
    return hipGetLastError();
}

} // namespace fgs
