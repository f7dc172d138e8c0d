// rows.cu -- row-wise operators around a layer: the residual addition with the
// root-mean-square norm (and an 8-bit copy of its result), and the widening of
// 8-bit rows.  Both move every byte once and are bound by HBM.
#include <cuda_fp8.h>

#include "ds4moe_internal.cuh"
#include "ops.cuh"

namespace ds4 {

namespace {

constexpr int kBlk = 256;   // columns a warp takes per step: 32 lanes x 8

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float round_bf16(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

// Eight consecutive elements at flat index i (16-byte aligned).
template <bool BF>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
    if constexpr (BF) {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(w[j]), v[2 * j + 1] = bf16_hi(w[j]);
    } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

__device__ __forceinline__ void store8(void* p, bool bf, int64_t i, const float (&v)[8]) {
    if (bf) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
            make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

template <bool BF>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (BF) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store1(void* p, bool bf, int64_t i, float v) {
    if (bf) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(p)[i] = v;
}

// One value as the code of the format: y / scale rounded to nearest even.  A
// scale of zero (an all-zero group) or NaN gives code 0.
__device__ __forceinline__ float quotient(float y, float scale) { return scale > 0.f ? __fdiv_rn(y, scale) : 0.f; }
__device__ __forceinline__ uint32_t code8(float t, int fmt) {
    if (fmt == kQ8E4M3) return __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)(uint8_t)(int8_t)max(-127, min(127, __float2int_rn(t)));   // NaN converts to 0
}
__device__ __forceinline__ uint32_t code8x2(float a, float b, int fmt) {
    if (fmt == kQ8E4M3) return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    return code8(a, fmt) | (code8(b, fmt) << 8);
}

}  // namespace

// A launch with its own status: what an earlier call of the thread left behind is
// not this launch's (a caller told of a failure would make the call again).
template <typename... P, typename... A>
static cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kernel, (P)args...);
}

// ---------------------------------------------------------------- residual addition and norm
// s = x + r (one binary32 add, rounded to r's type where that is stored);
// y = (s * rstd) * w with rstd = 1 / sqrt(mean(s^2) + eps); optionally y as
// 8-bit codes with one scale max|y| / qmax per group of columns.
//
// The row stays in registers between the two passes over it, so each input is
// read once.  The sum of squares is taken in binary64 (a product of two
// binary32 values is exact there) and rstd rounded to binary32 once: the
// result then does not depend on how the row is split over threads, down to
// the 8-bit codes next to a rounding border.  That costs one conversion and
// one binary64 FMA per element, about a sixth of the row's time in HBM.
//
// A warp takes blocks of 256 columns: eight consecutive columns per lane when
// rows are 16-byte aligned (VEC), else columns lane + 32 j.  The groups of
// 32, 64 or 128 columns of the scales lie inside a block either way.
template <bool XBF, int RT, int CH, bool VEC>   // RT: no residual 0, binary32 1, bf16 2
__global__ void __launch_bounds__(CH == 4 ? 512 : 1024) k_add_rmsnorm(AddNormArgs a) {
    __shared__ double s_sum[32];
    __shared__ uint32_t s_max[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const bool solo = a.warps_per_row == 1;
    const int64_t row = solo ? (int64_t)blockIdx.x * nw + warp : blockIdx.x;
    if (solo && row >= a.n) return;
    const int w0 = solo ? 0 : warp, W = a.warps_per_row;
    const int H = a.H;
    const int64_t base = row * H;

    // column of element e of this lane in block b
    auto col = [&](int b, int e) { return b * kBlk + (VEC ? lane * 8 + e : lane + 32 * e); };

    float s[CH][8];
    double acc = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int b = c * W + w0;
#pragma unroll
        for (int e = 0; e < 8; ++e) s[c][e] = 0.f;
        if constexpr (VEC) {
            if (col(b, 0) < H) load8<XBF>(a.x, base + col(b, 0), s[c]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col(b, e) < H) s[c][e] = load1<XBF>(a.x, base + col(b, e));
        }
    }
    if constexpr (RT != 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int b = c * W + w0;
            if constexpr (VEC) {
                if (col(b, 0) < H) {
                    float r[8];
                    load8<RT == 2>(a.res, base + col(b, 0), r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        s[c][e] = __fadd_rn(s[c][e], r[e]);
                        if constexpr (RT == 2) s[c][e] = round_bf16(s[c][e]);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col(b, e) < H) {
                        s[c][e] = __fadd_rn(s[c][e], load1<RT == 2>(a.res, base + col(b, e)));
                        if constexpr (RT == 2) s[c][e] = round_bf16(s[c][e]);
                    }
            }
        }
        // after every load: sum may be res itself
        if (a.sum) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int b = c * W + w0;
                if constexpr (VEC) {
                    if (col(b, 0) < H) store8(a.sum, RT == 2, base + col(b, 0), s[c]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col(b, e) < H) store1(a.sum, RT == 2, base + col(b, e), s[c][e]);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double d = (double)s[c][e];
            acc = fma(d, d, acc);
        }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    if (!solo) {
        if (lane == 0) s_sum[warp] = acc;
        __syncthreads();
        acc = 0.0;
        for (int i = 0; i < nw; ++i) acc += s_sum[i];
    }
    const float rstd = (float)rsqrt(fma(acc, a.inv_H, (double)a.eps));

    // y in place of s; the largest magnitude as its bit pattern (a NaN's is above infinity's, so it stays)
    uint32_t mx = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int b = c * W + w0;
        if constexpr (VEC) {
            if (col(b, 0) < H) {
                float w[8];
                load8<false>(a.w, col(b, 0), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[c][e] = __fmul_rn(__fmul_rn(s[c][e], rstd), w[e]);
                if (a.out) store8(a.out, a.out_bf16, base + col(b, 0), s[c]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) s[c][e] = 0.f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = col(b, e) < H;
                s[c][e] = in ? __fmul_rn(__fmul_rn(s[c][e], rstd), __ldg(a.w + col(b, e))) : 0.f;
                if (in && a.out) store1(a.out, a.out_bf16, base + col(b, e), s[c][e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = max(mx, __float_as_uint(s[c][e]) & 0x7fffffffu);
    }
    if (!a.q) return;

    float row_scale = 0.f;
    if (a.group == 0) {
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (!solo) {
            if (lane == 0) s_max[warp] = mx;
            __syncthreads();
            mx = 0;
            for (int i = 0; i < nw; ++i) mx = max(mx, s_max[i]);
        }
        row_scale = __fdiv_rn(__uint_as_float(mx), a.qmax);
        if (lane == 0 && w0 == 0) a.scale[row] = row_scale;
    }
    const int ngroups = a.group ? (H + a.group - 1) / a.group : 1;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int b = c * W + w0;
        if (b * kBlk >= H) break;
        if constexpr (VEC) {
            float sc = row_scale;
            if (a.group) {
                uint32_t g = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) g = max(g, __float_as_uint(s[c][e]) & 0x7fffffffu);
                g = max(g, __shfl_xor_sync(0xffffffffu, g, 1));   // 32 columns: four lanes
                g = max(g, __shfl_xor_sync(0xffffffffu, g, 2));
                if (a.group >= 64) g = max(g, __shfl_xor_sync(0xffffffffu, g, 4));
                if (a.group >= 128) g = max(g, __shfl_xor_sync(0xffffffffu, g, 8));
                sc = __fdiv_rn(__uint_as_float(g), a.qmax);
                if (lane % (a.group / 8) == 0 && col(b, 0) < H) a.scale[row * ngroups + col(b, 0) / a.group] = sc;
            }
            if (col(b, 0) < H) {
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = quotient(s[c][e], sc);
                const uint32_t lo = code8x2(t[0], t[1], a.fmt) | (code8x2(t[2], t[3], a.fmt) << 16);
                const uint32_t hi = code8x2(t[4], t[5], a.fmt) | (code8x2(t[6], t[7], a.fmt) << 16);
                *reinterpret_cast<uint2*>(a.q + base + col(b, 0)) = make_uint2(lo, hi);
            }
        } else {
            // columns 32 e .. 32 e + 31 of the block are element e of the 32 lanes
            uint32_t g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                g[e] = a.group ? __reduce_max_sync(0xffffffffu, __float_as_uint(s[c][e]) & 0x7fffffffu) : 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float sc = row_scale;
                if (a.group) {
                    uint32_t m = g[e];
                    if (a.group >= 64) m = max(m, g[e ^ 1]);
                    if (a.group >= 128) m = max(m, max(g[e ^ 2], g[e ^ 3]));
                    sc = __fdiv_rn(__uint_as_float(m), a.qmax);
                    if (lane == 0 && col(b, e) < H && (32 * e) % a.group == 0)
                        a.scale[row * ngroups + col(b, e) / a.group] = sc;
                }
                if (col(b, e) < H) a.q[base + col(b, e)] = (uint8_t)code8(quotient(s[c][e], sc), a.fmt);
            }
        }
    }
}

template <bool XBF, int RT, bool VEC>
static cudaError_t norm_launch(const AddNormArgs& a, int ch, dim3 grid, dim3 block, cudaStream_t st) {
    if (ch == 1) return launch(k_add_rmsnorm<XBF, RT, 1, VEC>, grid, block, st, a);
    if (ch == 2) return launch(k_add_rmsnorm<XBF, RT, 2, VEC>, grid, block, st, a);
    return launch(k_add_rmsnorm<XBF, RT, 4, VEC>, grid, block, st, a);
}

template <bool XBF, int RT>
static cudaError_t norm_launch_v(const AddNormArgs& a, bool vec, int ch, dim3 grid, dim3 block, cudaStream_t st) {
    return vec ? norm_launch<XBF, RT, true>(a, ch, grid, block, st) : norm_launch<XBF, RT, false>(a, ch, grid, block, st);
}

cudaError_t launch_add_rmsnorm(AddNormArgs a, bool x_bf16, int res_kind, bool vec, int n_sm, cudaStream_t st) {
    const int blocks = (a.H + kBlk - 1) / kBlk;
    // Few rows: one block per warp, the shortest chain.  Many: two, so that a
    // row's loads are in flight at once (4096 columns, 11,709 rows with every
    // output: 117 us; before a faster rstd 123, one block 156, four 145 us).  More than 32 blocks (8192
    // columns) need four to fit a CTA.
    int ch = blocks > 32 ? 4 : a.n < 2 * n_sm ? 1 : 2;
    if (blocks < ch) ch = 1;
    a.warps_per_row = (blocks + ch - 1) / ch;
    a.inv_H = 1.0 / (double)a.H;
    const bool solo = a.warps_per_row == 1;
    const int rows_per_cta = solo ? 4 : 1;
    const dim3 block(32 * (solo ? rows_per_cta : a.warps_per_row));
    const dim3 grid((unsigned)((a.n + rows_per_cta - 1) / rows_per_cta));
    if (x_bf16) {
        if (res_kind == 0) return norm_launch_v<true, 0>(a, vec, ch, grid, block, st);
        if (res_kind == 1) return norm_launch_v<true, 1>(a, vec, ch, grid, block, st);
        return norm_launch_v<true, 2>(a, vec, ch, grid, block, st);
    }
    if (res_kind == 0) return norm_launch_v<false, 0>(a, vec, ch, grid, block, st);
    if (res_kind == 1) return norm_launch_v<false, 1>(a, vec, ch, grid, block, st);
    return norm_launch_v<false, 2>(a, vec, ch, grid, block, st);
}

// ---------------------------------------------------------------- widening of 8-bit rows
// out = q * scale, one binary32 product (then one rounding where out is bf16).
// q and out are flat arrays with the same index, so a thread takes 16
// consecutive elements whatever the row width; only the scale's index follows
// rows and groups.
namespace {
__device__ __forceinline__ void widen4(uint32_t w, int fmt, float (&v)[4]) {
    if (fmt == kQ8E4M3) {
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        const float2 fa = __half22float2(__half2(a)), fb = __half22float2(__half2(b));
        v[0] = fa.x, v[1] = fa.y, v[2] = fb.x, v[3] = fb.y;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(uint8_t)(w >> (8 * j));
    }
}
}  // namespace

// I: the type of flat indices (32 bits where they suffice: the division by the
// row width costs as much as the rest otherwise).  A thread's pieces are in
// flight together: two where there are enough threads all the same (11,709 x
// 4096 to bf16: 24.0 us, one 32.5 us), one for few rows (61 x 2050 to binary32:
// 2.9 us, two 3.8 us).  Sixteen bf16 values are one 32-byte store, which needs a
// 32-byte address; out is 16-byte aligned (a view of rows may begin between),
// and then they are two stores.
template <bool OBF, typename I, int kWidenPieces>
__global__ void __launch_bounds__(256) k_widen_rows(const uint8_t* q, int fmt, const float* scale, int shift, int H,
                                                    I total, void* out) {
    const int ngroups = shift ? (H + (1 << shift) - 1) >> shift : 1;
    const bool out32 = ((uintptr_t)out & 31) == 0;   // the same for every piece of 32 bytes
    uint4 raw[kWidenPieces];
    float first[kWidenPieces];
    I row[kWidenPieces];
    int col[kWidenPieces];
#pragma unroll
    for (int p = 0; p < kWidenPieces; ++p) {
        const I i0 = ((I)blockIdx.x * (256 * kWidenPieces) + p * 256 + threadIdx.x) * 16;
        raw[p] = make_uint4(0, 0, 0, 0);
        row[p] = 0, col[p] = 0, first[p] = 0.f;
        if (i0 < total) {
            if (total - i0 >= 16) {
                raw[p] = ld_stream_v4(q + i0);
            } else {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < (int)(total - i0)) w[j >> 2] |= (uint32_t)q[i0 + j] << (8 * (j & 3));
                raw[p] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            row[p] = i0 / (I)H;
            col[p] = (int)(i0 - row[p] * (I)H);
            first[p] = __ldg(scale + (size_t)row[p] * ngroups + (shift ? col[p] >> shift : 0));
        }
    }
#pragma unroll
    for (int p = 0; p < kWidenPieces; ++p) {
        const I i0 = ((I)blockIdx.x * (256 * kWidenPieces) + p * 256 + threadIdx.x) * 16;
        if (i0 >= total) return;
        const int cnt = total - i0 < 16 ? (int)(total - i0) : 16;
        const uint32_t w[4] = {raw[p].x, raw[p].y, raw[p].z, raw[p].w};
        float v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float t[4];
            widen4(w[j], fmt, t);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * j + e] = t[e];
        }
        float sc = first[p];
        // columns up to the end of this scale's group
        int g = shift ? col[p] >> shift : 0;
        int left = (shift ? min(H, (g + 1) << shift) : H) - col[p];
        if (left >= cnt) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(v[j], sc);
        } else {
            size_t r = row[p];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (j < cnt) {
                    if (left == 0) {
                        if (++g == ngroups) g = 0, ++r;
                        sc = __ldg(scale + r * ngroups + g);
                        left = shift ? min(1 << shift, H - (g << shift)) : H;
                    }
                    v[j] = __fmul_rn(v[j], sc);
                    --left;
                }
            }
        }
        if (cnt == 16) {
            if constexpr (OBF) {
                uint32_t b[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) b[j] = bf16x2(v[2 * j], v[2 * j + 1]);
                uint16_t* o = static_cast<uint16_t*>(out) + i0;
                if (out32) {
                    st_global_v8(o, b[0], b[1], b[2], b[3], b[4], b[5], b[6], b[7]);
                } else {
                    reinterpret_cast<uint4*>(o)[0] = make_uint4(b[0], b[1], b[2], b[3]);
                    reinterpret_cast<uint4*>(o)[1] = make_uint4(b[4], b[5], b[6], b[7]);
                }
            } else {
                float* o = static_cast<float*>(out) + i0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    reinterpret_cast<float4*>(o)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j < cnt) store1(out, OBF, i0 + j, v[j]);
        }
    }
}

template <bool OBF, int P>
static cudaError_t widen_launch(const uint8_t* q, int fmt, const float* scale, int shift, int H, int64_t total, void* out,
                                cudaStream_t st) {
    const int64_t per = 256 * P * 16, ctas = (total + per - 1) / per;
    const dim3 grid((unsigned)ctas), block(256);
    if (ctas * per < ((int64_t)1 << 32))
        return launch(k_widen_rows<OBF, uint32_t, P>, grid, block, st, q, fmt, scale, shift, H, total, out);
    return launch(k_widen_rows<OBF, uint64_t, P>, grid, block, st, q, fmt, scale, shift, H, total, out);
}

cudaError_t launch_widen_rows(const uint8_t* q, int fmt, const float* scale, int group, int n, int H, void* out,
                              bool out_bf16, cudaStream_t st) {
    const int shift = group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : 0;
    const int64_t total = (int64_t)n * H;
    const bool few = total < ((int64_t)1 << 22);   // 1,024 CTAs of one piece per thread
    if (out_bf16)
        return few ? widen_launch<true, 1>(q, fmt, scale, shift, H, total, out, st)
                   : widen_launch<true, 2>(q, fmt, scale, shift, H, total, out, st);
    return few ? widen_launch<false, 1>(q, fmt, scale, shift, H, total, out, st)
               : widen_launch<false, 2>(q, fmt, scale, shift, H, total, out, st);
}

}  // namespace ds4
