// residual_norm.hip -- the boundary between two transformer blocks on gfx950:
// norm of the block's output, gate, scaled residual, norm for the next block,
// in one pass over the row, and its gradients.
//
//   z = y / rms(y) * w_post          (or y, without w_post)
//   r = alpha * x + gate * z         rounded to the residual's type
//   n = r / rms(r) * w_pre           of the rounded r
// with rms(t) = sqrt(mean(t^2) + eps), everything in FP32 between one read of
// each input and one rounding of each output.
//
// Backward, from what the forward pass kept (y, r) and the gradients dr, dn,
// with yh = y / rms(y), rh = r / rms(r):
//   d  = dr + (dn w_pre - rh mean(dn w_pre rh)) / rms(r)
//   dx = alpha d;  dgate = d z;  dz = d gate
//   dy = (dz w_post - yh mean(dz w_post yh)) / rms(y)     (or dz)
//   dw_pre = sum over rows of dn rh;  dw_post = sum over rows of dz yh
//
// Memory bounds both: a workgroup owns whole rows, held in registers, 8
// values a vector and VPT vectors a thread, and takes row after row so that
// the weights are read once; the next row's loads are issued before this
// row's sums.  Sums over rows stay in registers, one partial row a workgroup,
// and a second kernel adds the partial rows in a fixed order.
// Measured (a 2 GiB copy reaches 4.87 TB/s): forward 8192 x 16384, FP32
// residual, 302 us, 5.3 TB/s; backward 8192 x 4096, BF16 residual, 88 us,
// 4.6 TB/s with the sums' 5 us; backward 4111 x 7168, FP32 residual and a gate
// for each token, 135 us, 4.8 TB/s; backward rows of more than 8192 values
// reach 2.7 to 3.2 TB/s with a post norm (4096 x 16384, FP32, channel gate: 420
// us), where weights come from L2 for each row and 6 to 38 registers are
// spilled, and 4.4 to 4.8 with neither norm nor gate.
#include <algorithm>

#include "fgs_device.h"
#include "operators_internal.h"

namespace fgs {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <bool FP32> struct Raw { uint4 v[FP32 ? 2 : 1]; };   // 8 values as loaded

template <bool FP32>
__device__ __forceinline__ Raw<FP32> load8(const void* base, int64_t i)
{
    Raw<FP32> r;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + i * (FP32 ? 4 : 2));
    r.v[0] = p[0];
    if constexpr (FP32) r.v[1] = p[1];
    return r;
}
template <bool FP32>
__device__ __forceinline__ void unpack(const Raw<FP32>& r, float f[8])
{
    if constexpr (FP32) {
        f[0] = as_f32(r.v[0].x), f[1] = as_f32(r.v[0].y), f[2] = as_f32(r.v[0].z), f[3] = as_f32(r.v[0].w);
        f[4] = as_f32(r.v[1].x), f[5] = as_f32(r.v[1].y), f[6] = as_f32(r.v[1].z), f[7] = as_f32(r.v[1].w);
    } else {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const bf16x2 p = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, p);
}
template <bool FP32>
__device__ __forceinline__ void store8(void* base, int64_t i, const float f[8])
{
    uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + i * (FP32 ? 4 : 2));
    if constexpr (FP32) {
        p[0] = make_uint4(as_u32(f[0]), as_u32(f[1]), as_u32(f[2]), as_u32(f[3]));
        p[1] = make_uint4(as_u32(f[4]), as_u32(f[5]), as_u32(f[6]), as_u32(f[7]));
    } else {
        p[0] = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + as_f32((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u32(v), CTRL, 0xF, 0xF, false));
}
// the sum over the wave, in every lane
__device__ __forceinline__ float wave_sum(float v)
{
    v = dpp_add<DPP_XOR1>(v);
    v = dpp_add<DPP_XOR2>(v);
    v = dpp_add<DPP_HALF_MIRROR>(v);
    v = dpp_add<DPP_MIRROR>(v);
    auto a = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    v = as_f32(a[0]) + as_f32(a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return as_f32(b[0]) + as_f32(b[1]);
}
// N sums over the workgroup, in every thread.  `slots` alternates between two
// halves of the scratch from call to call, so one barrier a call is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* slots)
{
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
    const int waves = blockDim.x >> 6;
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) slots[k * 16 + (threadIdx.x >> 6)] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float s = 0.0f;
        for (int w = 0; w < waves; ++w) s += slots[k * 16 + w];
        v[k] = s;
    }
}

struct NormParams {
    const uint16_t* y;
    const void* x;          // forward: the residual; backward: r
    const float *w_post, *w_pre;
    const void* gate;
    const void* dr;
    const uint16_t* dn;
    void *r, *dx;
    uint16_t *n, *dy, *dgate;
    float *sum_pre, *sum_post, *sum_gate;   // the workgroups' partial rows, 3 W apart; one workgroup's are the results
    int64_t T, ldy, ldx, ldg, lddr, lddn;
    int W;
    int row_threads;        // backward: threads a row; a workgroup takes blockDim / row_threads rows at once
    float alpha, eps, inv_w;
};

enum { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_TOKEN = 2 };

template <int VPT, bool FP32, bool POST, int GATE>
__global__ __launch_bounds__(1024) void residual_norm_fwd_kernel(NormParams p)
{
    __shared__ float slots[2][16];
    const int vecs = p.W / 8, step = blockDim.x;
    float wpre[VPT][8], wpost[VPT][8], gch[VPT][8];
    Raw<false> y[VPT], gt[VPT];
    Raw<FP32> x[VPT];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * step;
            if (c >= vecs) break;
            y[j] = load8<false>(p.y, row * p.ldy + 8 * c);
            x[j] = load8<FP32>(p.x, row * p.ldx + 8 * c);
            if (GATE == GATE_TOKEN) gt[j] = load8<false>(p.gate, row * p.ldg + 8 * c);
        }
    };
    int64_t row = blockIdx.x;
    load(row);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + j * step;
        if (c >= vecs) break;
        unpack<true>(load8<true>(p.w_pre, 8 * c), wpre[j]);
        if (POST) unpack<true>(load8<true>(p.w_post, 8 * c), wpost[j]);
        if (GATE == GATE_CHANNEL) unpack<true>(load8<true>(p.gate, 8 * c), gch[j]);
    }
    for (; row < p.T; row += gridDim.x) {
        float z[VPT][8], xs[VPT][8], g[VPT][8];
        float sum[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if ((int)threadIdx.x + j * step >= vecs) break;
            unpack<false>(y[j], z[j]);
            unpack<FP32>(x[j], xs[j]);
            if (GATE == GATE_TOKEN) unpack<false>(gt[j], g[j]);
            if (POST)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(z[j][i], z[j][i], sum[0]);
        }
        if (row + gridDim.x < p.T) load(row + gridDim.x);
        float ry = 1.0f;
        if (POST) {
            block_sum(sum, slots[0]);
            ry = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], p.inv_w, p.eps));
        }
        sum[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * step;
            if (c >= vecs) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v = z[j][i];
                if (POST) v = v * ry * wpost[j][i];
                if (GATE == GATE_CHANNEL) v *= gch[j][i];
                if (GATE == GATE_TOKEN) v *= g[j][i];
                v = __builtin_fmaf(p.alpha, xs[j][i], v);
                // what is kept is what is normed
                if (!FP32) v = (float)(__bf16)v;
                z[j][i] = v;
                sum[0] = __builtin_fmaf(v, v, sum[0]);
            }
            store8<FP32>(p.r, row * p.W + 8 * c, z[j]);
        }
        block_sum(sum, slots[1]);
        const float rr = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], p.inv_w, p.eps));
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * step;
            if (c >= vecs) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) z[j][i] = z[j][i] * rr * wpre[j][i];
            store8<false>(p.n, row * p.W + 8 * c, z[j]);
        }
        // the next row's sums of y reuse slots[0]: with no barrier between
        // (POST off) a wave could still read slots[1] when it is written again
        if (!POST && blockDim.x > 64) __syncthreads();
    }
}

// Half h of 8 values as loaded.
template <bool FP32>
__device__ __forceinline__ void unpack4(const Raw<FP32>& r, int h, float f[4])
{
    if constexpr (FP32) {
        f[0] = as_f32(r.v[h].x), f[1] = as_f32(r.v[h].y), f[2] = as_f32(r.v[h].z), f[3] = as_f32(r.v[h].w);
    } else {
        const uint32_t a = h ? r.v[0].z : r.v[0].x, b = h ? r.v[0].w : r.v[0].y;
        f[0] = bf16_lo(a), f[1] = bf16_hi(a), f[2] = bf16_lo(b), f[3] = bf16_hi(b);
    }
}
template <bool FP32>
__device__ __forceinline__ void pack4(Raw<FP32>& r, int h, const float f[4])
{
    if constexpr (FP32) {
        r.v[h] = make_uint4(as_u32(f[0]), as_u32(f[1]), as_u32(f[2]), as_u32(f[3]));
    } else {
        (h ? r.v[0].z : r.v[0].x) = pack2(f[0], f[1]);
        (h ? r.v[0].w : r.v[0].y) = pack2(f[2], f[3]);
    }
}
// A row's address, the same in every lane, and 8 values of it by their 32-bit
// place: one scalar address a tensor instead of a vector one for each access.
template <bool FP32>
__device__ __forceinline__ char* row_of(const void* base, int64_t row, int64_t ld)
{
    return const_cast<char*>(static_cast<const char*>(base)) + row * ld * (FP32 ? 4 : 2);
}
template <bool FP32>
__device__ __forceinline__ Raw<FP32> load_at(const char* row, int c)
{
    Raw<FP32> r;
    const uint4* p = reinterpret_cast<const uint4*>(row + (uint32_t)(c * (FP32 ? 32 : 16)));
    r.v[0] = p[0];
    if constexpr (FP32) r.v[1] = p[1];
    return r;
}
template <bool FP32>
__device__ __forceinline__ void store_at(char* row, int c, const Raw<FP32>& r)
{
    uint4* p = reinterpret_cast<uint4*>(row + (uint32_t)(c * (FP32 ? 32 : 16)));
    p[0] = r.v[0];
    if constexpr (FP32) p[1] = r.v[1];
}
__device__ __forceinline__ void load4(const float* p, float f[4])
{
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}

// One barrier a row: with a = gate w_post y and b = dn w_pre, the sum that dy
// needs is linear in d,
//   sum a d = sum a dr + (sum a b - c1 / rms(r) sum a r) / rms(r),
// so all six row sums (r^2, b r, y^2 and these three) come from one pass over
// the row's registers, and the second pass writes every output.  The weights
// lie in LDS (read again for each row from L2 they cost more than the row
// itself: 8192 x 4096 with every option 102 us, and 4.1 against 5.1 TB/s for
// an FP32 residual), and the next row's loads are issued before this row's
// sums.  A workgroup fills a compute unit, so that 256 partial rows are all
// that the second kernel has to add; narrow rows go several at a time.
template <int VPT, bool FP32, bool POST, int GATE>
__global__ __launch_bounds__(1024) void residual_norm_bwd_kernel(NormParams p)
{
    // a wide row, two vectors a thread, needs the registers of two sums: LDS
    // holds these instead of the weights
    constexpr bool WIDE = VPT > 1;
    constexpr bool CHANNEL = GATE == GATE_CHANNEL;
    constexpr bool NEED_Y = POST || GATE != GATE_NONE;   // without a post norm, for the gate's gradient alone
    constexpr int SUMS = POST ? 6 : 2;
    extern __shared__ float4 lds4[];
    __shared__ float slots[2][6][16];
    float* lds = reinterpret_cast<float*>(lds4);
    const float* w_pre = WIDE ? p.w_pre : lds;
    const float* w_post = WIDE ? p.w_post : lds + p.W;
    const float* w_gate = WIDE ? static_cast<const float*>(p.gate) : lds + (POST ? 2 : 1) * p.W;
    float *wide_post = lds, *wide_gate = lds + (POST ? p.W : 0);

    const int vecs = p.W / 8, step = p.row_threads;
    const int waves = step >> 6, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = wave / waves, at_once = (int)(blockDim.x >> 6) / waves;
    const int c0 = threadIdx.x - slot * step;
    for (int i = threadIdx.x; i < p.W / 4; i += blockDim.x) {
        if (WIDE) {
            if (POST) lds4[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (CHANNEL) lds4[(POST ? p.W / 4 : 0) + i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            continue;
        }
        lds4[i] = reinterpret_cast<const float4*>(p.w_pre)[i];
        if (POST) lds4[p.W / 4 + i] = reinterpret_cast<const float4*>(p.w_post)[i];
        if (CHANNEL) lds4[(POST ? 2 : 1) * (p.W / 4) + i] = reinterpret_cast<const float4*>(p.gate)[i];
    }

    struct Row { Raw<false> y[VPT], dn[VPT], g[VPT]; Raw<FP32> r[VPT], dr[VPT]; };
    auto load = [&](Row& to, int64_t row) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = c0 + j * step;
            if (c >= vecs || row >= p.T) break;
            to.r[j] = load_at<FP32>(row_of<FP32>(p.x, row, p.ldx), c);
            to.dn[j] = load_at<false>(row_of<false>(p.dn, row, p.lddn), c);
            if (NEED_Y) to.y[j] = load_at<false>(row_of<false>(p.y, row, p.ldy), c);
            to.dr[j] = load_at<FP32>(row_of<FP32>(p.dr, row, p.lddr), c);
            if (GATE == GATE_TOKEN) to.g[j] = load_at<false>(row_of<false>(p.gate, row, p.ldg), c);
        }
    };
    auto gate_of = [&](const Row& now, int j, int c, int h, float g[4]) {
        if (GATE == GATE_TOKEN) unpack4<false>(now.g[j], h, g);
        else if (CHANNEL) load4(w_gate + (uint32_t)(8 * c + 4 * h), g);
    };
    float a_pre[VPT][8], a_post[VPT][8], a_gate[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) a_pre[j][i] = a_post[j][i] = a_gate[j][i] = 0.0f;
    auto to_lds = [](float* at, const float f[4]) { *reinterpret_cast<float4*>(at) = make_float4(f[0], f[1], f[2], f[3]); };

    auto one = [&](Row& now, int64_t row, int parity) {
        float sum[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = c0 + j * step;
            if (c >= vecs || row >= p.T) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[4], r[4], b[4], y[4], wp[4], g[4], dr[4];
                load4(w_pre + (uint32_t)(8 * c + 4 * h), w);
                unpack4<FP32>(now.r[j], h, r);
                unpack4<false>(now.dn[j], h, b);
                if (POST) {
                    unpack4<false>(now.y[j], h, y);
                    load4(w_post + (uint32_t)(8 * c + 4 * h), wp);
                    unpack4<FP32>(now.dr[j], h, dr);
                    gate_of(now, j, c, h, g);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    b[i] *= w[i];
                    sum[0] = __builtin_fmaf(r[i], r[i], sum[0]);
                    sum[1] = __builtin_fmaf(b[i], r[i], sum[1]);
                    if (POST) {
                        const float a = GATE == GATE_NONE ? wp[i] * y[i] : g[i] * wp[i] * y[i];
                        sum[2] = __builtin_fmaf(y[i], y[i], sum[2]);
                        sum[3] = __builtin_fmaf(a, dr[i], sum[3]);
                        sum[4] = __builtin_fmaf(a, b[i], sum[4]);
                        sum[5] = __builtin_fmaf(a, r[i], sum[5]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int k = 0; k < SUMS; ++k) sum[k] = wave_sum(sum[k]);
        if (waves > 1) {
            // slots alternate from row to row, so one barrier is enough
            if (lane == 0)
#pragma unroll
                for (int k = 0; k < SUMS; ++k) slots[parity][k][wave] = sum[k];
            __syncthreads();
            const int w = lane & 15;
#pragma unroll
            for (int k = 0; k < SUMS; ++k) {
                float v = w < waves ? slots[parity][k][slot * waves + w] : 0.0f;
                v = dpp_add<DPP_XOR1>(v);
                v = dpp_add<DPP_XOR2>(v);
                v = dpp_add<DPP_HALF_MIRROR>(v);
                sum[k] = dpp_add<DPP_MIRROR>(v);
            }
        }
        if (row >= p.T) return;
        const float rr = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], p.inv_w, p.eps));
        const float c1 = sum[1] * rr * p.inv_w;
        const float ry = POST ? __builtin_amdgcn_rsqf(__builtin_fmaf(sum[2], p.inv_w, p.eps)) : 1.0f;
        const float c2 = POST ? (sum[3] + rr * (sum[4] - c1 * rr * sum[5])) * ry * p.inv_w : 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = c0 + j * step;
            if (c >= vecs) break;
            // two vectors of every input, sums and outputs pass 128 registers:
            // the gate is read again, and with every option on FP32 rows are
            // (4096 x 16384: 449 -> 417 us; without a gate 315 -> 345, so there not)
            if (WIDE && FP32 && POST && GATE != GATE_NONE) {
                now.r[j] = load_at<FP32>(row_of<FP32>(p.x, row, p.ldx), c);
                now.dr[j] = load_at<FP32>(row_of<FP32>(p.dr, row, p.lddr), c);
            }
            if (WIDE && GATE == GATE_TOKEN) now.g[j] = load_at<false>(row_of<false>(p.gate, row, p.ldg), c);
            Raw<FP32> dx_out;
            Raw<false> dy_out, dg_out;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[4], r[4], dn[4], y[4], wp[4], g[4], d[4], dg[4], dy[4];
                load4(w_pre + (uint32_t)(8 * c + 4 * h), w);
                if (POST) load4(w_post + (uint32_t)(8 * c + 4 * h), wp);
                unpack4<FP32>(now.r[j], h, r);
                unpack4<false>(now.dn[j], h, dn);
                unpack4<FP32>(now.dr[j], h, d);
                if (NEED_Y) unpack4<false>(now.y[j], h, y);
                gate_of(now, j, c, h, g);
                float *sum_post = a_post[j] + 4 * h, *sum_gate = a_gate[j] + 4 * h;
                float wide_p[4], wide_g[4];
                if (WIDE && POST) load4(wide_post + (uint32_t)(8 * c + 4 * h), sum_post = wide_p);
                if (WIDE && CHANNEL) load4(wide_gate + (uint32_t)(8 * c + 4 * h), sum_gate = wide_g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float rh = r[i] * rr;
                    a_pre[j][4 * h + i] = __builtin_fmaf(dn[i], rh, a_pre[j][4 * h + i]);
                    const float dd = __builtin_fmaf(rr, __builtin_fmaf(-rh, c1, dn[i] * w[i]), d[i]);
                    d[i] = p.alpha * dd;
                    const float yh = POST ? y[i] * ry : 0.0f;
                    if (GATE != GATE_NONE) {
                        const float z = POST ? yh * wp[i] : y[i];
                        if (CHANNEL) sum_gate[i] = __builtin_fmaf(dd, z, sum_gate[i]);
                        else dg[i] = dd * z;
                    }
                    float dz = GATE == GATE_NONE ? dd : dd * g[i];
                    if (POST) {
                        sum_post[i] = __builtin_fmaf(dz, yh, sum_post[i]);
                        dz = ry * __builtin_fmaf(-yh, c2, dz * wp[i]);
                    }
                    dy[i] = dz;
                }
                if (WIDE && POST) to_lds(wide_post + (uint32_t)(8 * c + 4 * h), wide_p);
                if (WIDE && CHANNEL) to_lds(wide_gate + (uint32_t)(8 * c + 4 * h), wide_g);
                pack4<FP32>(dx_out, h, d);
                pack4<false>(dy_out, h, dy);
                if (GATE == GATE_TOKEN) pack4<false>(dg_out, h, dg);
                __builtin_amdgcn_sched_barrier(0);
            }
            store_at<FP32>(row_of<FP32>(p.dx, row, p.W), c, dx_out);
            store_at<false>(row_of<false>(p.dy, row, p.W), c, dy_out);
            if (GATE == GATE_TOKEN) store_at<false>(row_of<false>(p.dgate, row, p.W), c, dg_out);
        }
    };

    // every wave of the workgroup takes as many turns, with or without a row
    const int64_t stride = (int64_t)gridDim.x * at_once;
    int64_t first = (int64_t)blockIdx.x * at_once;
    int parity = 0;
    Row now, next;
    load(now, first + slot);
    __syncthreads();
    for (; first < p.T; first += stride) {
        if constexpr (VPT == 1) {
            load(next, first + stride + slot);
            one(now, first + slot, parity);
            now = next;
        } else {
            one(now, first + slot, parity);
            load(now, first + stride + slot);
        }
        parity ^= 1;
    }
    // the rows' sums, slot after slot through LDS
    for (int s = 1; s < at_once; ++s) {
        __syncthreads();
        if (slot == s && c0 < vecs) {
            store8<true>(lds, 8 * c0, a_pre[0]);
            if (POST) store8<true>(lds, p.W + 8 * c0, a_post[0]);
            if (CHANNEL) store8<true>(lds, (POST ? 2 : 1) * p.W + 8 * c0, a_gate[0]);
        }
        __syncthreads();
        if (slot == 0 && c0 < vecs) {
            float f[8];
            unpack<true>(load8<true>(lds, 8 * c0), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) a_pre[0][i] += f[i];
            if (POST) {
                unpack<true>(load8<true>(lds, p.W + 8 * c0), f);
#pragma unroll
                for (int i = 0; i < 8; ++i) a_post[0][i] += f[i];
            }
            if (CHANNEL) {
                unpack<true>(load8<true>(lds, (POST ? 2 : 1) * p.W + 8 * c0), f);
#pragma unroll
                for (int i = 0; i < 8; ++i) a_gate[0][i] += f[i];
            }
        }
    }
    if (slot != 0) return;
    const int64_t out = (int64_t)blockIdx.x * 3 * p.W;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = c0 + j * step;
        if (c >= vecs) break;
        if (WIDE && POST) unpack<true>(load8<true>(wide_post, 8 * c), a_post[j]);
        if (WIDE && CHANNEL) unpack<true>(load8<true>(wide_gate, 8 * c), a_gate[j]);
        store8<true>(p.sum_pre, out + 8 * c, a_pre[j]);
        if (POST) store8<true>(p.sum_post, out + 8 * c, a_post[j]);
        if (CHANNEL) store8<true>(p.sum_gate, out + 8 * c, a_gate[j]);
    }
}

// The partial rows of a column added in a fixed order: 32 columns a workgroup,
// 8 threads of 4 columns, 32 rows at once and 8 loads in flight a thread, then
// the 32 sums in order.
__global__ __launch_bounds__(256) void residual_norm_sum_kernel(const float* partial, int parts, int W, float* dw_pre,
                                                                float* dw_post, float* dgate)
{
    __shared__ float s[32][33];
    float* out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
    if (!out) return;
    const int col = 4 * (threadIdx.x & 7), lane = threadIdx.x >> 3;
    const int c = blockIdx.x * 32 + col;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < W) {
        const float* at = partial + (int64_t)blockIdx.y * W + c;
        for (int i = lane; i < parts; i += 8 * 32) {
            float4 x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = i + 32 * k < parts ? *reinterpret_cast<const float4*>(at + (int64_t)(i + 32 * k) * 3 * W)
                                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[0] += x[k].x, v[1] += x[k].y, v[2] += x[k].z, v[3] += x[k].w;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) s[lane][col + k] = v[k];
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < W) {
        float t = 0.0f;
        for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
        out[blockIdx.x * 32 + threadIdx.x] = t;
    }
}

// Vectors a thread, and threads a workgroup.
struct Shape { int vpt, threads; };
Shape shape_of(int W, int most)
{
    const int vecs = W / 8;
    const int vpt = vecs <= most ? 1 : 2;
    return {vpt, ((vecs + vpt - 1) / vpt + 63) / 64 * 64};
}
constexpr int FWD_SINGLE = 64, BWD_SINGLE = 1024;    // vectors up to which a thread has one

template <bool FWD, int VPT, bool FP32, bool POST, int GATE>
void launch_one(const NormParams& p, int grid, int threads, hipStream_t stream)
{
    if constexpr (FWD)
        residual_norm_fwd_kernel<VPT, FP32, POST, GATE><<<grid, threads, 0, stream>>>(p);
    else
        residual_norm_bwd_kernel<VPT, FP32, POST, GATE><<<
            grid, threads, ((VPT == 1) + POST + (GATE == GATE_CHANNEL)) * p.W * sizeof(float), stream>>>(p);
}
template <bool FWD, int VPT, bool FP32, bool POST>
void launch_gate(const NormParams& p, int gate, int grid, int threads, hipStream_t stream)
{
    if (gate == GATE_NONE) launch_one<FWD, VPT, FP32, POST, GATE_NONE>(p, grid, threads, stream);
    else if (gate == GATE_CHANNEL) launch_one<FWD, VPT, FP32, POST, GATE_CHANNEL>(p, grid, threads, stream);
    else launch_one<FWD, VPT, FP32, POST, GATE_TOKEN>(p, grid, threads, stream);
}
template <bool FWD, int VPT>
void launch_types(const NormParams& p, const NormArgs& a, int grid, int threads, hipStream_t stream)
{
    if (a.fp32 && a.w_post) launch_gate<FWD, VPT, true, true>(p, a.gate_kind, grid, threads, stream);
    else if (a.fp32) launch_gate<FWD, VPT, true, false>(p, a.gate_kind, grid, threads, stream);
    else if (a.w_post) launch_gate<FWD, VPT, false, true>(p, a.gate_kind, grid, threads, stream);
    else launch_gate<FWD, VPT, false, false>(p, a.gate_kind, grid, threads, stream);
}

NormParams params(const NormArgs& a)
{
    NormParams p{};
    p.y = (const uint16_t*)a.y, p.x = a.x, p.w_post = a.w_post, p.w_pre = a.w_pre, p.gate = a.gate;
    p.dr = a.dr, p.dn = (const uint16_t*)a.dn;
    p.r = a.r, p.n = (uint16_t*)a.n, p.dx = a.dx, p.dy = (uint16_t*)a.dy, p.dgate = (uint16_t*)a.dgate;
    p.T = a.T, p.W = (int)a.W, p.ldy = a.ldy, p.ldx = a.ldx, p.ldg = a.ldg, p.lddr = a.lddr, p.lddn = a.lddn;
    p.alpha = a.alpha, p.eps = a.eps, p.inv_w = 1.0f / (float)a.W;
    return p;
}

} // namespace

// The backward kernel's workgroups, one partial row each: one a compute unit,
// of as many rows at once as 1024 threads hold and the rows give it.  Rows that
// one workgroup holds at once need no second kernel, whose launch takes the
// host as long as theirs does (a call of 7 x 512: 21.9 -> 19.1 us).
namespace {
struct BwdShape { int vpt, row_threads, at_once, grid; };
BwdShape bwd_shape(int64_t T, int64_t W)
{
    const Shape s = shape_of((int)W, BWD_SINGLE);
    BwdShape b{s.vpt, s.threads, 1, 0};
    const int64_t most = 1024 / s.threads;
    b.at_once = (int)std::max<int64_t>(1, T <= most ? T : std::min<int64_t>(most, T / 256));
    b.grid = (int)std::min<int64_t>((T + b.at_once - 1) / b.at_once, 256);
    return b;
}
} // namespace
int residual_norm_parts(int64_t T, int64_t W) { return bwd_shape(T, W).grid; }

hipError_t launch_residual_norm_fwd(const NormArgs& a, hipStream_t stream)
{
    const NormParams p = params(a);
    const Shape s = shape_of((int)a.W, FWD_SINGLE);
    const int grid = (int)std::min<int64_t>(a.T, (int64_t)device_cus() * std::max(2, 1536 / s.threads));
    if (s.vpt == 1) launch_types<true, 1>(p, a, grid, s.threads, stream);
    else launch_types<true, 2>(p, a, grid, s.threads, stream);       // 16384 values: 1024 threads
    return hipGetLastError();
}

hipError_t launch_residual_norm_bwd(const NormArgs& a, hipStream_t stream)
{
    NormParams p = params(a);
    const BwdShape s = bwd_shape(a.T, a.W);
    p.row_threads = s.row_threads;
    // (with an aligned place for the kernel's 16-byte stores)
    const bool direct = s.grid == 1 &&
                        (((uintptr_t)a.dw_pre | (a.w_post ? (uintptr_t)a.dw_post : 0) |
                          (a.gate_kind == GATE_CHANNEL ? (uintptr_t)a.dgate : 0)) & 15) == 0;
    p.sum_pre = direct ? a.dw_pre : a.partial;
    p.sum_post = direct ? a.dw_post : a.partial + a.W;
    p.sum_gate = direct ? (float*)a.dgate : a.partial + 2 * a.W;
    if (s.grid > 0) {
        if (s.vpt == 1) launch_types<false, 1>(p, a, s.grid, s.row_threads * s.at_once, stream);
        else launch_types<false, 2>(p, a, s.grid, s.row_threads, stream);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || direct) return e;
    residual_norm_sum_kernel<<<dim3((unsigned)((a.W + 31) / 32), 3), 256, 0, stream>>>(
        a.partial, s.grid, (int)a.W, a.dw_pre, a.w_post ? a.dw_post : nullptr,
        a.gate_kind == GATE_CHANNEL ? (float*)a.dgate : nullptr);
    return hipGetLastError();
}

} // namespace fgs
