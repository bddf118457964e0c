// norm_kernels.h -- the norms before and after a block (gfx950).
//
//   residual norm: r = residual + scale * x,  out = r * inv * w
//   gated norm:    v = y * silu(z),           out = v * inv * w   (or v = y and out = v * inv * w * silu(z))
// with inv = 1 / sqrt(mean(v^2) + eps) over a row (or a group of its channels).
//
// All of them move each element once and are bound by that: a row lives in
// registers between its reduction and its outputs.  THREADS threads take a row
// (64: a wave, four rows to a workgroup; 256 or 1024: the workgroup), each of
// them VPT vectors of 8 channels.  Sums are fp32.
//
// Backward, with e = w * dout (times silu(z) where the norm is before the gate):
//     dv = inv * (e - v * inv^2 * mean(e v))
// from one reduction of sum v^2 and sum e v together.  The sums over rows for
// the parameters stay in registers while a workgroup walks over its rows, go
// to the workspace once, and are added up there in row order.
#pragma once

#include "block_device.h"

namespace ss {

struct NormParams {
    const void *x, *res, *dout, *dres_out;   // x: the scan's y for the gated norm; res: also the stored residual in backward
    const void* z;
    const float *scale, *w;
    void *out, *res_out, *dx, *dres, *dz;
    float* part;          // (parts, d) shares of dweight, then of dscale
    int64_t rows, d;      // d: channels of a whole row
    int64_t xs, zs;       // row strides of x (or y) and z
    int gd, groups;       // channels normalised together, and how many such groups a row has
    int parts;            // shares per channel
    float eps;
    int before;
};

__device__ __forceinline__ f32x8 load8(const float* p) {
    const f32x4 a = __builtin_bit_cast(f32x4, load16(p)), b = __builtin_bit_cast(f32x4, load16(p + 4));
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ f32x8 load8(const uint16_t* p) {
    return Mat<uint16_t>::unpack(__builtin_bit_cast(bf16x8, load16(p)));
}
__device__ __forceinline__ void store8(float* p, f32x8 v) {
    store16(p, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
    store16(p + 4, __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}));
}
__device__ __forceinline__ void store8(uint16_t* p, f32x8 v) {
    store16(p, __builtin_bit_cast(u32x4, Mat<uint16_t>::pack(v)));
}

// The channels of one of a row's THREADS threads: vectors of 8, the last one
// of a row perhaps partly beyond its gd channels.
template <int THREADS>
struct Lanes {
    static __device__ __forceinline__ int at(int k) { return (int(threadIdx.x) % THREADS + THREADS * k) * 8; }
    template <typename T>
    static __device__ __forceinline__ f32x8 load(const T* p, int k, int gd) {
        f32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
        if (at(k) + 8 <= gd) {
            v = load8(p + at(k));
        } else if (at(k) < gd) {
#pragma unroll
            for (int e = 0; e < 7; e++)
                if (at(k) + e < gd) v[e] = Elem<T>::load(p, at(k) + e);
        }
        return v;
    }
    template <typename T>
    static __device__ __forceinline__ void store(T* p, int k, int gd, f32x8 v) {
        if (at(k) + 8 <= gd) {
            store8(p + at(k), v);
        } else if (at(k) < gd) {
#pragma unroll
            for (int e = 0; e < 7; e++)
                if (at(k) + e < gd) Elem<T>::store(p, at(k) + e, v[e]);
        }
    }
};

// Sums of a and b over the THREADS threads of a row, in every one of them.
template <int THREADS>
__device__ __forceinline__ void row_sums(float& a, float& b, float* red) {
    a = sum_wave(a);
    b = sum_wave(b);
    if constexpr (THREADS > 64) {
        constexpr int W = THREADS / 64;
        const int wave = int(threadIdx.x) >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
            red[wave] = a;
            red[W + wave] = b;
        }
        __syncthreads();
        a = red[0];
        b = red[W];
#pragma unroll
        for (int i = 1; i < W; i++) {
            a += red[i];
            b += red[W + i];
        }
    }
}

__device__ __forceinline__ float inv_rms(float sum_sq, int n, float eps) {
    return __builtin_amdgcn_rsqf(sum_sq / float(n) + eps);
}

// residual + scale * x with the product rounded first, as two operations do.
__device__ __forceinline__ float scaled_sum(float res, float x, float scale) {
#pragma clang fp contract(off)
    const float sx = scale * x;
    return res + sx;
}

// A value as it is stored in type T.
template <typename T>
__device__ __forceinline__ float stored(float v) { return widen(narrow<T>(v)); }

template <typename T, typename TR, int THREADS, int VPT>
__global__ __launch_bounds__(THREADS > 256 ? THREADS : 256) void residual_norm_fwd(NormParams p) {
    using Ln = Lanes<THREADS>;
    constexpr int RPW = THREADS == 64 ? 4 : 1;   // rows per workgroup
    __shared__ float red[2 * (THREADS > 64 ? THREADS / 64 : 1)];
    const int gd = p.gd;
    for (int64_t row = int64_t(blockIdx.x) * RPW + threadIdx.x / THREADS; row < p.rows; row += int64_t(gridDim.x) * RPW) {
        f32x8 r[VPT];
        float sq = 0.0f, unused = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            const f32x8 x = Ln::load(static_cast<const T*>(p.x) + row * p.xs, k, gd);
            f32x8 v = x;
            if (p.scale || p.res) {
                f32x8 res = {0, 0, 0, 0, 0, 0, 0, 0}, sc = {1, 1, 1, 1, 1, 1, 1, 1};
                if (p.res) res = Ln::load(static_cast<const TR*>(p.res) + row * p.d, k, gd);
                if (p.scale) sc = Ln::load(p.scale, k, gd);
#pragma unroll
                for (int e = 0; e < 8; e++) v[e] = scaled_sum(res[e], x[e], sc[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; e++) {
                v[e] = stored<TR>(v[e]);
                sq += v[e] * v[e];
            }
            r[k] = v;
            Ln::store(static_cast<TR*>(p.res_out) + row * p.d, k, gd, v);
        }
        row_sums<THREADS>(sq, unused, red);
        const float inv = inv_rms(sq, gd, p.eps);
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            const f32x8 w = Ln::load(p.w, k, gd);
            Ln::store(static_cast<T*>(p.out) + row * p.d, k, gd, r[k] * inv * w);
        }
    }
}

template <typename T, typename TR, int THREADS, int VPT>
__global__ __launch_bounds__(THREADS > 256 ? THREADS : 256) void residual_norm_bwd(NormParams p) {
    using Ln = Lanes<THREADS>;
    constexpr int RPW = THREADS == 64 ? 4 : 1;
    __shared__ float red[2 * (THREADS > 64 ? THREADS / 64 : 1)];
    const int gd = p.gd;
    const int part = int(blockIdx.x) * RPW + int(threadIdx.x) / THREADS;
    if (part >= p.parts) return;   // whole waves of a workgroup whose rows share nothing
    f32x8 dw[VPT], ds[VPT];
#pragma unroll
    for (int k = 0; k < VPT; k++) dw[k] = ds[k] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t row = part; row < p.rows; row += p.parts) {
        f32x8 r[VPT], g[VPT];
        float sq = 0.0f, ev = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            r[k] = Ln::load(static_cast<const TR*>(p.res) + row * p.d, k, gd);
            g[k] = Ln::load(static_cast<const T*>(p.dout) + row * p.d, k, gd);
            const f32x8 w = Ln::load(p.w, k, gd);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                sq += r[k][e] * r[k][e];
                ev += g[k][e] * w[e] * r[k][e];
            }
        }
        row_sums<THREADS>(sq, ev, red);
        const float inv = inv_rms(sq, gd, p.eps), coef = inv * inv * (ev / float(gd));
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            const f32x8 w = Ln::load(p.w, k, gd);
            f32x8 dr = {0, 0, 0, 0, 0, 0, 0, 0};
            if (p.dres_out) dr = Ln::load(static_cast<const TR*>(p.dres_out) + row * p.d, k, gd);
            dr += (g[k] * w - r[k] * coef) * inv;
            dw[k] += g[k] * r[k] * inv;
            if (p.dres) Ln::store(static_cast<TR*>(p.dres) + row * p.d, k, gd, dr);
            if (p.scale) {
                ds[k] += dr * Ln::load(static_cast<const T*>(p.x) + row * p.xs, k, gd);
                dr *= Ln::load(p.scale, k, gd);
            }
            Ln::store(static_cast<T*>(p.dx) + row * p.d, k, gd, dr);
        }
    }
    float* const to = p.part + int64_t(part) * p.d;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
        Ln::store(to, k, gd, dw[k]);
        if (p.scale) Ln::store(to + int64_t(p.parts) * p.d, k, gd, ds[k]);
    }
}

__device__ __forceinline__ float sigmoid(float z) { return rcp_hw(1.0f + exp2_hw(-z * kLog2e)); }

template <typename T, int THREADS, int VPT>
__global__ __launch_bounds__(THREADS > 256 ? THREADS : 256) void gated_norm_fwd(NormParams p) {
    using Ln = Lanes<THREADS>;
    constexpr int RPW = THREADS == 64 ? 4 : 1;
    __shared__ float red[2 * (THREADS > 64 ? THREADS / 64 : 1)];
    const int gd = p.gd;
    for (int64_t at = int64_t(blockIdx.x) * RPW + threadIdx.x / THREADS; at < p.rows * p.groups;
         at += int64_t(gridDim.x) * RPW) {
        const int64_t row = at / p.groups;
        const int c0 = int(at % p.groups) * gd;   // the group's first channel
        f32x8 v[VPT], gate[VPT];
        float sq = 0.0f, unused = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            v[k] = Ln::load(static_cast<const T*>(p.x) + row * p.xs + c0, k, gd);
            gate[k] = Ln::load(static_cast<const T*>(p.z) + row * p.zs + c0, k, gd);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                gate[k][e] *= sigmoid(gate[k][e]);
                if (!p.before) v[k][e] *= gate[k][e];
                sq += v[k][e] * v[k][e];
            }
        }
        row_sums<THREADS>(sq, unused, red);
        const float inv = inv_rms(sq, gd, p.eps);
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            f32x8 o = v[k] * inv * Ln::load(p.w + c0, k, gd);
            if (p.before) o *= gate[k];
            Ln::store(static_cast<T*>(p.out) + row * p.d + c0, k, gd, o);
        }
    }
}

template <typename T, int THREADS, int VPT>
__global__ __launch_bounds__(THREADS > 256 ? THREADS : 256) void gated_norm_bwd(NormParams p) {
    using Ln = Lanes<THREADS>;
    constexpr int RPW = THREADS == 64 ? 4 : 1;
    __shared__ float red[2 * (THREADS > 64 ? THREADS / 64 : 1)];
    const int gd = p.gd;
    const int64_t unit = int64_t(blockIdx.x) * RPW + threadIdx.x / THREADS;
    if (unit >= int64_t(p.parts) * p.groups) return;
    const int part = int(unit / p.groups), c0 = int(unit % p.groups) * gd;
    f32x8 dw[VPT];
#pragma unroll
    for (int k = 0; k < VPT; k++) dw[k] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t row = part; row < p.rows; row += p.parts) {
        f32x8 y[VPT], z[VPT], g[VPT];
        float sq = 0.0f, ev = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            y[k] = Ln::load(static_cast<const T*>(p.x) + row * p.xs + c0, k, gd);
            z[k] = Ln::load(static_cast<const T*>(p.z) + row * p.zs + c0, k, gd);
            g[k] = Ln::load(static_cast<const T*>(p.dout) + row * p.d + c0, k, gd);
            const f32x8 w = Ln::load(p.w + c0, k, gd);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float gate = z[k][e] * sigmoid(z[k][e]);
                const float v = p.before ? y[k][e] : y[k][e] * gate;
                const float en = p.before ? g[k][e] * w[e] * gate : g[k][e] * w[e];
                sq += v * v;
                ev += en * v;
            }
        }
        row_sums<THREADS>(sq, ev, red);
        const float inv = inv_rms(sq, gd, p.eps), coef = inv * inv * (ev / float(gd));
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            const f32x8 w = Ln::load(p.w + c0, k, gd);
            f32x8 dy, dz;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float sg = sigmoid(z[k][e]), gate = z[k][e] * sg;
                const float slope = sg + gate * (1.0f - sg);   // d silu / dz
                const float v = p.before ? y[k][e] : y[k][e] * gate;
                const float en = p.before ? g[k][e] * w[e] * gate : g[k][e] * w[e];
                const float dv = inv * (en - v * coef);
                const float hat = v * inv;
                dy[e] = p.before ? dv : dv * gate;
                dz[e] = (p.before ? g[k][e] * hat * w[e] : dv * y[k][e]) * slope;
                dw[k][e] += p.before ? g[k][e] * gate * hat : g[k][e] * hat;
            }
            Ln::store(static_cast<T*>(p.dx) + row * p.d + c0, k, gd, dy);
            Ln::store(static_cast<T*>(p.dz) + row * p.d + c0, k, gd, dz);
        }
    }
#pragma unroll
    for (int k = 0; k < VPT; k++) Ln::store(p.part + int64_t(part) * p.d + c0, k, gd, dw[k]);
}

// out[c] = sum over the parts of src[part][c]: 64 channels and 16 shares of the
// parts to a workgroup, each share in part order, then the shares in order.
// blockIdx.y picks dweight or dscale.
__global__ __launch_bounds__(1024) void norm_sum_parts(const float* src, float* dweight, float* dscale, int parts,
                                                       int64_t d) {
    __shared__ float share[16][64];
    const int64_t c = int64_t(blockIdx.x) * 64 + (threadIdx.x & 63);
    const int s = int(threadIdx.x) >> 6;
    if (blockIdx.y == 1) src += int64_t(parts) * d;
    float v = 0.0f;
    if (c < d)
        for (int i = s; i < parts; i += 16) v += src[int64_t(i) * d + c];
    share[s][threadIdx.x & 63] = v;
    __syncthreads();
    if (s == 0 && c < d) {
#pragma unroll
        for (int i = 1; i < 16; i++) v += share[i][threadIdx.x];
        (blockIdx.y == 1 ? dscale : dweight)[c] = v;
    }
}

}  // namespace ss
