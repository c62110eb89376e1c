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
#include <algorithm>

#include "fgs_device.h"
#include "fgs_internal.h"

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
    float* partial;         // [workgroups][3][W]: dw_pre, dw_post, dgate
    int64_t T, ldy, ldx, ldg, lddr, lddn;
    int W;
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

template <int VPT, bool FP32, bool POST, int GATE>
__global__ __launch_bounds__(512) void residual_norm_bwd_kernel(NormParams p)
{
    __shared__ float slots[2][3 * 16];
    const int vecs = p.W / 8, step = blockDim.x;
    float a_pre[VPT][8], a_post[VPT][8], a_gate[VPT][8];
    Raw<false> y[VPT], dn[VPT], gt[VPT];
    Raw<FP32> r[VPT], dr[VPT];
    // without a post norm, y is needed for the gate's gradient alone
    constexpr bool NEED_Y = POST || GATE != GATE_NONE;
    auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * step;
            if (c >= vecs) break;
            if (NEED_Y) y[j] = load8<false>(p.y, row * p.ldy + 8 * c);
            r[j] = load8<FP32>(p.x, row * p.ldx + 8 * c);
            dn[j] = load8<false>(p.dn, row * p.lddn + 8 * c);
            dr[j] = load8<FP32>(p.dr, row * p.lddr + 8 * c);
            if (GATE == GATE_TOKEN) gt[j] = load8<false>(p.gate, row * p.ldg + 8 * c);
        }
    };
    int64_t row = blockIdx.x;
    load(row);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) a_pre[j][i] = a_post[j][i] = a_gate[j][i] = 0.0f;
    for (; row < p.T; row += gridDim.x) {
        float sum[3] = {0.0f, 0.0f, 0.0f};      // r^2, dn w_pre r, y^2
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * step;
            if (c >= vecs) break;
            float w[8], f[8], d[8], v[8];
            unpack<true>(load8<true>(p.w_pre, 8 * c), w);
            unpack<FP32>(r[j], f);
            unpack<false>(dn[j], d);
            if (POST) unpack<false>(y[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[0] = __builtin_fmaf(f[i], f[i], sum[0]);
                sum[1] = __builtin_fmaf(d[i] * w[i], f[i], sum[1]);
                if (POST) sum[2] = __builtin_fmaf(v[i], v[i], sum[2]);
            }
        }
        block_sum(sum, slots[0]);
        const float rr = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], p.inv_w, p.eps));
        const float c1 = sum[1] * rr * p.inv_w;
        const float ry = POST ? __builtin_amdgcn_rsqf(__builtin_fmaf(sum[2], p.inv_w, p.eps)) : 1.0f;
        float t[VPT][8], sum2[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * step;
            if (c >= vecs) break;
            float w[8], f[8], d[8], v[8], g[8], wp[8], dx[8];
            unpack<true>(load8<true>(p.w_pre, 8 * c), w);
            unpack<FP32>(r[j], f);
            unpack<false>(dn[j], d);
            unpack<FP32>(dr[j], dx);
            if (NEED_Y) unpack<false>(y[j], v);
            if (POST) unpack<true>(load8<true>(p.w_post, 8 * c), wp);
            if (GATE == GATE_CHANNEL) unpack<true>(load8<true>(p.gate, 8 * c), g);
            if (GATE == GATE_TOKEN) unpack<false>(gt[j], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float fh = f[i] * rr;
                a_pre[j][i] = __builtin_fmaf(d[i], fh, a_pre[j][i]);
                const float dd = __builtin_fmaf(rr, __builtin_fmaf(-fh, c1, d[i] * w[i]), dx[i]);
                dx[i] = p.alpha * dd;
                const float yh = POST ? v[i] * ry : 0.0f;
                if (GATE != GATE_NONE) {
                    const float dg = dd * (POST ? yh * wp[i] : v[i]);
                    if (GATE == GATE_CHANNEL) a_gate[j][i] += dg;
                    else f[i] = dg;
                }
                float dz = GATE == GATE_NONE ? dd : dd * g[i];
                if (POST) {
                    a_post[j][i] = __builtin_fmaf(dz, yh, a_post[j][i]);
                    dz *= wp[i];
                    sum2[0] = __builtin_fmaf(dz, v[i], sum2[0]);
                }
                t[j][i] = dz;
            }
            store8<FP32>(p.dx, row * p.W + 8 * c, dx);
            if (GATE == GATE_TOKEN) store8<false>(p.dgate, row * p.W + 8 * c, f);
        }
        float c2 = 0.0f;
        if (POST) {
            block_sum(sum2, slots[1]);
            c2 = sum2[0] * ry * p.inv_w;
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * step;
            if (c >= vecs) break;
            if (POST) {
                float v[8];
                unpack<false>(y[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) t[j][i] = ry * __builtin_fmaf(-v[i] * ry, c2, t[j][i]);
            }
            store8<false>(p.dy, row * p.W + 8 * c, t[j]);
        }
        if (row + gridDim.x < p.T) load(row + gridDim.x);
        if (!POST && blockDim.x > 64) __syncthreads();
    }
    float* out = p.partial + (int64_t)blockIdx.x * 3 * p.W;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + j * step;
        if (c >= vecs) break;
        store8<true>(out, 8 * c, a_pre[j]);
        if (POST) store8<true>(out, p.W + 8 * c, a_post[j]);
        if (GATE == GATE_CHANNEL) store8<true>(out, 2 * p.W + 8 * c, a_gate[j]);
    }
}

// The partial rows of a column added in order: 16 threads a column, 16
// columns a workgroup, then their 16 sums in order.
__global__ __launch_bounds__(256) void residual_norm_sum_kernel(const float* partial, int parts, int W, float* dw_pre,
                                                                float* dw_post, float* dgate)
{
    __shared__ float s[16][17];
    float* out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
    if (!out) return;
    const int col = threadIdx.x & 15, lane = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + col;
    float v = 0.0f;
    if (c < W)
        for (int i = lane; i < parts; i += 16) v += partial[((int64_t)i * 3 + blockIdx.y) * W + c];
    s[lane][col] = v;
    __syncthreads();
    if (lane == 0 && c < W) {
        v = 0.0f;
        for (int i = 0; i < 16; ++i) v += s[i][col];
        out[c] = v;
    }
}

// Vectors a thread, and threads: the fewest vectors that leave at most
// `most` threads a row.
struct Shape { int vpt, threads; };
Shape shape_of(int W, int most)
{
    const int vecs = W / 8;
    int vpt = vecs <= 64 ? 1 : 2;
    while (vpt < 4 && (vecs + vpt - 1) / vpt > most) vpt *= 2;
    const int threads = (vecs + vpt - 1) / vpt;
    return {vpt, std::max(64, (threads + 63) / 64 * 64)};
}

template <bool FWD, int VPT, bool FP32, bool POST, int GATE>
void launch_one(const NormParams& p, int grid, int threads, hipStream_t stream)
{
    if constexpr (FWD)
        residual_norm_fwd_kernel<VPT, FP32, POST, GATE><<<grid, threads, 0, stream>>>(p);
    else
        residual_norm_bwd_kernel<VPT, FP32, POST, GATE><<<grid, threads, 0, stream>>>(p);
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
    p.partial = a.partial;
    p.T = a.T, p.W = (int)a.W, p.ldy = a.ldy, p.ldx = a.ldx, p.ldg = a.ldg, p.lddr = a.lddr, p.lddn = a.lddn;
    p.alpha = a.alpha, p.eps = a.eps, p.inv_w = 1.0f / (float)a.W;
    return p;
}

} // namespace

// Workgroups of the backward kernel, one partial row each: two a compute
// unit, more where they are small.
int residual_norm_parts(int64_t T, int64_t W)
{
    const Shape s = shape_of((int)W, 512);
    return (int)std::min<int64_t>(T, (int64_t)256 * std::max(2, 512 / s.threads));
}

hipError_t launch_residual_norm_fwd(const NormArgs& a, hipStream_t stream)
{
    const NormParams p = params(a);
    const Shape s = shape_of((int)a.W, 1024);
    const int grid = (int)std::min<int64_t>(a.T, (int64_t)device_cus() * std::max(2, 1536 / s.threads));
    if (s.vpt == 1) launch_types<true, 1>(p, a, grid, s.threads, stream);
    else launch_types<true, 2>(p, a, grid, s.threads, stream);       // 16384 values: 1024 threads
    return hipGetLastError();
}

hipError_t launch_residual_norm_bwd(const NormArgs& a, hipStream_t stream)
{
    const NormParams p = params(a);
    const Shape s = shape_of((int)a.W, 512);
    const int grid = residual_norm_parts(a.T, a.W);
    if (grid > 0) {
        if (s.vpt == 1) launch_types<false, 1>(p, a, grid, s.threads, stream);
        else if (s.vpt == 2) launch_types<false, 2>(p, a, grid, s.threads, stream);
        else launch_types<false, 4>(p, a, grid, s.threads, stream);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    residual_norm_sum_kernel<<<dim3((unsigned)((a.W + 15) / 16), 3), 256, 0, stream>>>(
        a.partial, grid, (int)a.W, a.dw_pre, a.w_post ? a.dw_post : nullptr,
        a.gate_kind == GATE_CHANNEL ? (float*)a.dgate : nullptr);
    return hipGetLastError();
}

} // namespace fgs
