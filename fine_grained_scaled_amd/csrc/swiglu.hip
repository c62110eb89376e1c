// swiglu.hip -- SwiGLU with its input kept in 8 bits for the backward pass, on
// gfx950.
//
//   h = g sigmoid(g) u                 of gate_up = [g | u], rounded to BF16
//   dg = dh u sigmoid(g) (1 + g (1 - sigmoid(g))),  du = dh g sigmoid(g)
//
// The forward pass keeps g and u as E4M3 codes with one FP32 scale for each
// 128 values of a row, the library's 1x128 quantization (the last tile of a half
// may be shorter), two bytes a pair instead of four; the backward pass takes
// the gradients at the values that the codes stand for.  Both are one pass over
// their data, bound by memory: 4 bytes in, 2 + 2 out a pair forward, 2 + 2 in, 4
// out backward.
//
// Sixteen lanes take one tile of one row, 8 values of each half a lane; a
// workgroup takes four neighbouring tiles of four rows, which reads and writes
// 1 KiB of a row at a time (one tile of 16 rows, 256 bytes at a time, is slower
// though it writes the scales, [tile][row], 64 bytes at a time: 8192 x 14336
// forward and backward 349 us against 315, 6.0 TB/s; 4111 x 5464 85 against 69;
// two or four rows a thread 358 and 368).
#include <algorithm>

#include "fgs_device.h"
#include "operators_internal.h"

namespace fgs {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int TILES = 4, ROWS = 16 / TILES;      // a workgroup's tiles and rows
constexpr float LOG2E = 1.44269504088896340736f;

__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// sigmoid(g) = root^2 one and 1 - sigmoid(g) = rest, within a few FP32 steps.
// The factors are products of two with the root on each side, so that neither
// underflows before the product does where they are alike: exp(-|g|) alone leaves
// FP32's normal numbers at 87.  one (and the slope) go to the first of the two,
// so that nothing overflows before the product does.
__device__ __forceinline__ void sigmoid(float g, float& root, float& one, float& rest)
{
    const float t = __builtin_amdgcn_exp2f(-__builtin_fabsf(g) * (0.5f * LOG2E)), e = t * t;
    one = __builtin_amdgcn_rcpf(1.0f + e);
    root = g >= 0.0f ? 1.0f : t;
    rest = g >= 0.0f ? e * one : one;
}

__device__ __forceinline__ void unpack(const uint4& v, float f[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
}
__device__ __forceinline__ uint4 pack(const float f[8])
{
    return make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7]));
}

// The codes of a lane's 8 values of a tile held by 16 lanes, and the tile's scale.
__device__ __forceinline__ uint2 quantize(const uint4& v, float& scale)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    const E4M3Block b = e4m3_block_from_amax_bits(max_lanes16(top));
    scale = b.s;
    if (b.nan) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[2 * i] = e4m3_quotient_bits(w[i] << 16, b);
        q[2 * i + 1] = e4m3_quotient_bits(w[i] & 0xFFFF0000u, b);
    }
    return make_uint2(e4m3_pack4(q[0], q[1], q[2], q[3]), e4m3_pack4(q[4], q[5], q[6], q[7]));
}

template <bool KEEP>
__global__ __launch_bounds__(256) void swiglu_fwd_kernel(SwigluArgs p)
{
    const int lane = threadIdx.x & 15;
    const int at = threadIdx.x >> 4;
    const uint32_t across = (uint32_t)((p.I + 128 * TILES - 1) / (128 * TILES)), down = blockIdx.x / across;
    const int64_t row = (int64_t)down * ROWS + at / TILES, tile = (int64_t)(blockIdx.x - down * across) * TILES + at % TILES;
    const int64_t col = 128 * tile + 8 * lane;
    const bool in = row < p.T && col < p.I;
    uint4 g = {}, u = {};
    if (in) {
        const uint16_t* from = static_cast<const uint16_t*>(p.gate_up) + row * p.ld + col;
        g = *reinterpret_cast<const uint4*>(from);
        u = *reinterpret_cast<const uint4*>(from + p.I);
        float a[8], b[8];
        unpack(g, a);
        unpack(u, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float root, one, rest;
            sigmoid(a[k], root, one, rest);
            a[k] = (a[k] * root * one) * (b[k] * root);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h) + row * p.I + col) = pack(a);
    }
    if constexpr (KEEP) {
        float sg, su;
        const uint2 cg = quantize(g, sg), cu = quantize(u, su);
        if (in) {
            uint8_t* to = p.q + row * 2 * p.I + col;
            *reinterpret_cast<uint2*>(to) = cg;
            *reinterpret_cast<uint2*>(to + p.I) = cu;
            if (lane == 0) {
                const int64_t tiles = (p.I + 127) / 128;
                p.scales[tile * p.T + row] = sg;
                p.scales[(tiles + tile) * p.T + row] = su;
            }
        }
    }
}

// The values of 8 codes times their scale (a NaN scale has NaN codes).
__device__ __forceinline__ void decode(const uint2& c, float scale, float f[8])
{
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        f[4 * i] = a[0] * scale, f[4 * i + 1] = a[1] * scale, f[4 * i + 2] = b[0] * scale, f[4 * i + 3] = b[1] * scale;
    }
}

template <bool KEPT>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(SwigluArgs p)
{
    const int lane = threadIdx.x & 15;
    const int at = threadIdx.x >> 4;
    const uint32_t across = (uint32_t)((p.I + 128 * TILES - 1) / (128 * TILES)), down = blockIdx.x / across;
    const int64_t row = (int64_t)down * ROWS + at / TILES, tile = (int64_t)(blockIdx.x - down * across) * TILES + at % TILES;
    const int64_t col = 128 * tile + 8 * lane;
    if (row >= p.T || col >= p.I) return;
    float g[8], u[8], d[8];
    unpack(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.dh) + row * p.ldh + col), d);
    if constexpr (KEPT) {
        const uint8_t* from = p.q + row * 2 * p.I + col;
        const int64_t tiles = (p.I + 127) / 128;
        decode(*reinterpret_cast<const uint2*>(from), p.scales[tile * p.T + row], g);
        decode(*reinterpret_cast<const uint2*>(from + p.I), p.scales[(tiles + tile) * p.T + row], u);
    } else {
        const uint16_t* from = static_cast<const uint16_t*>(p.gate_up) + row * p.ld + col;
        unpack(*reinterpret_cast<const uint4*>(from), g);
        unpack(*reinterpret_cast<const uint4*>(from + p.I), u);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float root, one, rest;
        sigmoid(g[k], root, one, rest);
        const float ds = d[k] * root * one;
        const float dg = (ds * __builtin_fmaf(g[k], rest, 1.0f)) * (u[k] * root);
        u[k] = ds * (g[k] * root);
        g[k] = dg;
    }
    uint16_t* to = static_cast<uint16_t*>(p.dgate_up) + row * 2 * p.I + col;
    *reinterpret_cast<uint4*>(to) = pack(g);
    *reinterpret_cast<uint4*>(to + p.I) = pack(u);
}

uint32_t grid_of(const SwigluArgs& a) { return (uint32_t)swiglu_blocks(a.T, a.I); }

} // namespace

int64_t swiglu_blocks(int64_t T, int64_t I) { return (T + ROWS - 1) / ROWS * ((I + 128 * TILES - 1) / (128 * TILES)); }

hipError_t launch_swiglu_fwd(const SwigluArgs& a, hipStream_t stream)
{
    (a.q ? swiglu_fwd_kernel<true> : swiglu_fwd_kernel<false>)<<<grid_of(a), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwigluArgs& a, hipStream_t stream)
{
    (a.q ? swiglu_bwd_kernel<true> : swiglu_bwd_kernel<false>)<<<grid_of(a), 256, 0, stream>>>(a);
    return hipGetLastError();
}

} // namespace fgs
