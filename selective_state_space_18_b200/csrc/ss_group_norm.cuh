// ss_group_norm.cuh -- group norm of each row's channels, with an activation or a gate.
//
// Per row and group of `size` consecutive channels (a head of a state-space layer's
// output, say):
//   x' = gate_first ? x silu(gate) : x
//   n  = (x' - m) / sqrt(mean((x' - m)^2) + eps),  m = mean(x') (0 when not centred)
//   n  = n * weight + bias;  n = silu(n) when activated
//   y  = gate given and not gate_first ? n silu(gate) : n
// Statistics in fp32 from the values in registers, the mean first and then the squared
// distances from it (no difference of large sums).
//
// Bound by HBM: x and the gate are read once and y is written once.  A group is held in
// the registers of a team of lanes: 2^k lanes of a warp when it fits into 32 lanes of NV
// vectors, a whole CTA of 256 threads otherwise.  Vectors are 16 bytes where the group
// size and every row allow it (VEC elements), single elements elsewhere.
#pragma once

#include "ss_device.cuh"

namespace ss {

constexpr int kGnThreads = 256;
enum { kGnCenter = 1, kGnGateFirst = 2, kGnSilu = 4, kGnShared = 8 };

struct GroupNormArgs {
    int64_t rows;
    int groups, size; // channels = groups * size
    const void *x, *gate;
    int64_t x_stride, gate_stride; // elements between consecutive rows
    const float *weight, *bias;    // [channels], or [size] with kGnShared; nullable
    void *y;                       // [rows, channels]
    float eps, inv_size;
    int mode;      // kGn* bits
    int team_log2; // lanes of a warp per group (warp teams)
};

template <typename T, int VEC> struct GnVec;
template <typename T> struct GnVec<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = Elem<T>::load_smem(&v); }
    static __device__ __forceinline__ void store(T *p, const float (&f)[1]) { Elem<T>::store(p, f[0]); }
};
template <> struct GnVec<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float *p) { v = __ldcs(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w; }
    static __device__ __forceinline__ void store(float *p, const float (&f)[4])
    {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
    }
};
template <> struct GnVec<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[8])
    {
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                        pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
    }
};

template <int VEC> __device__ __forceinline__ void gn_params(const float *p, int i, float (&f)[VEC])
{
    if constexpr (VEC == 1) {
        f[0] = __ldg(p + i);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(p + i + e));
            f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
        }
    }
}

// Sum over the team: 2^team_log2 lanes of a warp, or all threads of the CTA.
template <bool CTA> __device__ __forceinline__ float gn_sum(float v, int team_log2, float *red)
{
    if constexpr (CTA) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        __syncthreads(); // the previous sum has been read
        if ((threadIdx.x & 31) == 0)
            red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < kGnThreads / 32; ++w)
            v += red[w];
        return v;
    } else {
        for (int o = (1 << team_log2) >> 1; o; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
}

// One group per team and turn; teams take groups grid-strided.
template <typename T, int VEC, int NV, bool CTA>
__global__ void __launch_bounds__(kGnThreads) ss_group_norm_kernel(const GroupNormArgs a)
{
    __shared__ float red[kGnThreads / 32];
    const int team = CTA ? kGnThreads : 1 << a.team_log2;
    const int per_cta = kGnThreads / team, lane = threadIdx.x & (team - 1);
    const int64_t total = a.rows * a.groups;
    const int64_t step = int64_t(gridDim.x) * per_cta;
    // every lane of a warp makes the same number of turns (the sums are warp-collective)
    for (int64_t first = int64_t(blockIdx.x) * per_cta; first < total; first += step) {
        const int64_t item = first + threadIdx.x / team;
        const bool live = item < total;
        const int64_t row = live ? item / a.groups : 0;
        const int grp = live ? int(item - row * a.groups) : 0;
        const T *xp = static_cast<const T *>(a.x) + row * a.x_stride + int64_t(grp) * a.size;
        const T *zp = a.gate ? static_cast<const T *>(a.gate) + row * a.gate_stride + int64_t(grp) * a.size : nullptr;
        float x[NV][VEC];
        GnVec<T, VEC> zv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = VEC * (lane + team * i);
            GnVec<T, VEC> xv;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                x[i][e] = 0.0f;
            if (live && c < a.size) {
                xv.load(xp + c);
                if (zp)
                    zv[i].load(zp + c);
                xv.get(x[i]);
            }
        }
        if (zp && (a.mode & kGnGateFirst)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (live && VEC * (lane + team * i) < a.size) {
                    float z[VEC];
                    zv[i].get(z);
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        x[i][e] *= silu(z[e]);
                }
            }
        }
        float mean = 0.0f;
        if (a.mode & kGnCenter) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    s += x[i][e];
            mean = gn_sum<CTA>(s, a.team_log2, red) * a.inv_size;
        }
        float s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (VEC * (lane + team * i) < a.size) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    x[i][e] -= mean;
                    s2 = fmaf(x[i][e], x[i][e], s2);
                }
            }
        }
        const float rs = rsqrtf(gn_sum<CTA>(s2, a.team_log2, red) * a.inv_size + a.eps);
        if (!live)
            continue;
        T *yp = static_cast<T *>(a.y) + (row * a.groups + grp) * a.size;
        const int pofs = (a.mode & kGnShared) ? 0 : grp * a.size;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = VEC * (lane + team * i);
            if (c >= a.size)
                break;
            float o[VEC], w[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                o[e] = x[i][e] * rs;
            if (a.weight) {
                gn_params<VEC>(a.weight, pofs + c, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    o[e] *= w[e];
            }
            if (a.bias) {
                gn_params<VEC>(a.bias, pofs + c, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    o[e] += w[e];
            }
            if (a.mode & kGnSilu) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    o[e] = silu(o[e]);
            }
            if (zp && !(a.mode & kGnGateFirst)) {
                zv[i].get(w);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    o[e] *= silu(w[e]);
            }
            GnVec<T, VEC>::store(yp + c, o);
        }
    }
}

} // namespace ss
