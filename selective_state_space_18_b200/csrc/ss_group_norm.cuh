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
// the registers of a team of lanes: 2^k lanes of a warp when it fits into 32 lanes of up
// to eight vectors, a whole CTA of 256 threads otherwise.  Vectors are 16 bytes where the group
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

// silu of a pair: v / (1 + 2^(-v log2 e)), with the reciprocal of the hardware (1 ulp; of
// infinity it is 0, so large negative v give -0).
__device__ __forceinline__ float2 gn_silu2(float2 v)
{
    const float2 t = __fmul2_rn(v, make_float2(-kLog2e, -kLog2e));
    const float2 d = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.0f, 1.0f));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    return __fmul2_rn(v, r);
}

// CTAs per SM to ask for, by the elements a lane holds: the loads in flight are what hides
// the memory's latency, and a lane has one vector per 8 (or 4) of its elements in flight.
__host__ __device__ constexpr int gn_min_ctas(int elements)
{
    return elements <= 8 ? 6 : elements <= 16 ? 4 : elements <= 24 ? 3 : elements <= 40 ? 2 : 1;
}

// One group per team and turn; teams take groups grid-strided.  A lane's elements are held
// and worked on as pairs (packed fp32 arithmetic: two elements an instruction); the
// instructions per element are what a group of many small rows is bound by.
// FULL: the group fills its team's vectors, so that nothing is guarded (with the guards
// 16384 x 32 groups of 128 took 75 us, a third of their instructions being guards).
// Measured: 70 us for 16384 x 32 groups of 128 bf16 with a gate (403 MB moved, 5.7 TB/s, 88% of
// a copy's rate), 33 us for 4096 x 8 groups of 640 fp32 (168 MB, 5.1 TB/s).
template <typename T, int VEC, int NV, bool CTA, bool FULL>
__global__ void __launch_bounds__(kGnThreads, gn_min_ctas(NV * VEC)) ss_group_norm_kernel(const GroupNormArgs a)
{
    constexpr int kE = NV * VEC, kP = (kE + 1) / 2; // elements and pairs of a lane
    __shared__ float red[kGnThreads / 32];
    const int team = CTA ? kGnThreads : 1 << a.team_log2;
    const int per_cta = kGnThreads / team, lane = threadIdx.x & (team - 1);
    const int64_t total = a.rows * a.groups;
    const int64_t step = int64_t(gridDim.x) * per_cta;
    // (row, group) of the team's item, advanced without divisions
    const int64_t row_step = step / a.groups;
    const int grp_step = int(step - row_step * a.groups);
    int64_t item = int64_t(blockIdx.x) * per_cta + threadIdx.x / team;
    int64_t row = item / a.groups;
    int grp = int(item - row * a.groups);
    const bool gated = a.gate != nullptr, gate_first = gated && (a.mode & kGnGateFirst);
    const int c0 = VEC * lane; // this lane's first element; its vectors are VEC * team apart
    auto in = [&](int i) { return FULL || c0 + VEC * team * i < a.size; }; // vector i is in the group
    // every lane of a warp makes the same number of turns (the sums are warp-collective)
    for (int64_t first = int64_t(blockIdx.x) * per_cta; first < total; first += step) {
        const bool live = item < total; // (teams past the end repeat the last group, unstored)
        if (!live) {
            row = a.rows - 1;
            grp = a.groups - 1;
        }
        const int64_t at = row * a.x_stride + int64_t(grp) * a.size;
        GnVec<T, VEC> xv[NV], zv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i))
                xv[i].load(static_cast<const T *>(a.x) + at + c0 + VEC * team * i);
        if (gated) {
            const int64_t zat = row * a.gate_stride + int64_t(grp) * a.size;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in(i))
                    zv[i].load(static_cast<const T *>(a.gate) + zat + c0 + VEC * team * i);
        }
        float2 x[kP];
        auto unpack = [&](const GnVec<T, VEC> (&raw)[NV], float2 (&f)[kP]) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    v[e] = 0.0f;
                if (in(i))
                    raw[i].get(v);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    ((VEC * i + e) & 1 ? f[(VEC * i + e) / 2].y : f[(VEC * i + e) / 2].x) = v[e];
            }
            if constexpr (kE & 1)
                f[kP - 1].y = 0.0f;
        };
        unpack(xv, x);
        if (gate_first) {
            float2 z[kP];
            unpack(zv, z);
#pragma unroll
            for (int p = 0; p < kP; ++p)
                x[p] = __fmul2_rn(x[p], gn_silu2(z[p]));
        }
        if (a.mode & kGnCenter) {
            float2 s = x[0];
#pragma unroll
            for (int p = 1; p < kP; ++p)
                s = __fadd2_rn(s, x[p]);
            const float mean = gn_sum<CTA>(s.x + s.y, a.team_log2, red) * a.inv_size;
#pragma unroll
            for (int e = 0; e < kE; ++e) { // (elements beyond the group stay 0)
                float &f = e & 1 ? x[e / 2].y : x[e / 2].x;
                f = in(e / VEC) ? f - mean : 0.0f;
            }
        }
        float2 s2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
        for (int p = 1; p < kP; ++p)
            s2 = __ffma2_rn(x[p], x[p], s2);
        const float rs = rsqrtf(gn_sum<CTA>(s2.x + s2.y, a.team_log2, red) * a.inv_size + a.eps);
#pragma unroll
        for (int p = 0; p < kP; ++p)
            x[p] = __fmul2_rn(x[p], make_float2(rs, rs));
        const int pofs = ((a.mode & kGnShared) ? 0 : grp * a.size) + c0;
        auto params = [&](const float *src, float2 (&f)[kP]) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    v[e] = 0.0f;
                if (in(i))
                    gn_params<VEC>(src, pofs + VEC * team * i, v);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    ((VEC * i + e) & 1 ? f[(VEC * i + e) / 2].y : f[(VEC * i + e) / 2].x) = v[e];
            }
            if constexpr (kE & 1)
                f[kP - 1].y = 0.0f;
        };
        if (a.weight) {
            float2 w[kP];
            params(a.weight, w);
#pragma unroll
            for (int p = 0; p < kP; ++p)
                x[p] = __fmul2_rn(x[p], w[p]);
        }
        if (a.bias) {
            float2 w[kP];
            params(a.bias, w);
#pragma unroll
            for (int p = 0; p < kP; ++p)
                x[p] = __fadd2_rn(x[p], w[p]);
        }
        if (a.mode & kGnSilu) {
#pragma unroll
            for (int p = 0; p < kP; ++p)
                x[p] = gn_silu2(x[p]);
        }
        if (gated && !gate_first) {
            float2 z[kP];
            unpack(zv, z);
#pragma unroll
            for (int p = 0; p < kP; ++p)
                x[p] = __fmul2_rn(x[p], gn_silu2(z[p]));
        }
        T *yp = static_cast<T *>(a.y) + (row * a.groups + grp) * a.size + c0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (live && in(i)) {
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    o[e] = (VEC * i + e) & 1 ? x[(VEC * i + e) / 2].y : x[(VEC * i + e) / 2].x;
                GnVec<T, VEC>::store(yp + VEC * team * i, o);
            }
        }
        item += step;
        row += row_step;
        grp += grp_step;
        if (grp >= a.groups) {
            grp -= a.groups;
            ++row;
        }
    }
}

} // namespace ss
