// ss_delta.cuh -- the gated delta rule: the prompt scan token by token, and the
// single-token decode step.
//
// Per batch row and value head h (which reads query / key head h / (heads_v / heads_k)),
// with the state S [dk x dv] in fp32, a_t = exp(g_t) (0 where the state is reset):
//   u_t = beta_t (v_t - a_t S_{t-1}^T k_t)
//   S_t = a_t S_{t-1} + k_t u_t^T
//   y_t = scale S_t^T q_t = scale (a_t S_{t-1}^T q_t + (q_t . k_t) u_t)
// (the write removes what the key reads already).  The last form reads the same old
// state as u_t, so one pass over S gives both dot products.  With SS_QK_L2NORM, q and k
// stand for q / sqrt(|q|^2 + eps) and k / sqrt(|k|^2 + eps).
#pragma once

#include "ss_device.cuh"

namespace ss {

constexpr float kDeltaEps = 1e-6f; // inside the square root of the q / k norms

struct DeltaArgs {
    int64_t batch, seq;
    int heads_k, heads_v, ratio, dk, dv; // ratio = heads_v / heads_k
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride; // elements between consecutive tokens
    const float *g, *beta;                // [batch, seq, heads_v], nullable: 0 and 1
    const uint8_t *reset;                 // [batch, seq], nullable
    const float *h0;                      // [batch, heads_v, dk, dv], nullable
    void *y;                              // [batch, seq, heads_v, dv]
    float *final_state;                   // [batch, heads_v, dk, dv], nullable
    float scale;
    int l2norm;
};

// ---- prompt scan, token by token -----------------------------------------------------
//
// A CTA owns one (batch row, value head) and 16 of its value columns: columns of the
// state never meet.  Four consumer warps hold the state in registers, a column's dk rows
// over 8 lanes; eight producer warps stage the next 16 tokens, two each (q and k in fp32,
// normalised and scaled, zero-padded to the kernel's dk; v; the decay, beta and q . k),
// while the consumers walk the current ones.  Per token a consumer lane reads its 4 R4 rows of k
// and q with 16-byte loads (four columns of a warp share each), and the two dot products
// are reduced over the 8 lanes together.  What bounds it is the latency of that chain,
// token after token, so it serves fp32 storage, key sizes the chunked form does not take
// and prompts of a few tokens; all its arithmetic is fp32.

constexpr int kDrCols = 16, kDrTok = 16, kDrConsumers = 128, kDrProducers = 256;
constexpr int kDrThreads = kDrConsumers + kDrProducers;

template <int R4> struct DeltaRecSmem { // floats of one staging buffer
    static constexpr int kDk = 32 * R4; // padded key size
    static constexpr int kK = 0, kQ = kDrTok * kDk, kV = 2 * kDrTok * kDk, kS = kV + kDrTok * kDrCols;
    static constexpr int kFloats = kS + 4 * kDrTok; // per token: decay, beta, q . k, (unused)
    static constexpr size_t kBytes = 2 * size_t(kFloats) * 4;
};

template <typename T, int R4>
__global__ void __launch_bounds__(kDrThreads) ss_delta_rec_kernel(const DeltaArgs a)
{
    using Sm = DeltaRecSmem<R4>;
    extern __shared__ __align__(16) float dr_sm[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int tiles = (a.dv + kDrCols - 1) / kDrCols;
    const int c0 = int(blockIdx.x % tiles) * kDrCols;
    const int64_t bh = blockIdx.x / tiles;
    const int64_t b = bh / a.heads_v;
    const int h = int(bh % a.heads_v), hk = h / a.ratio;
    const int64_t tok0 = b * a.seq; // first token of this batch row
    const int64_t ntiles = (a.seq + kDrTok - 1) / kDrTok;

    // producer warp w stages tokens w and w + 8 of a tile, the loads of both in flight together
    auto stage = [&](int64_t tile, float *buf) {
        constexpr int kPer = kDrTok / (kDrProducers / 32);
        const int w = (tid - kDrConsumers) >> 5;
        float q[kPer][R4], k[kPer][R4], v[kPer], g[kPer], be[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int64_t pos = tile * kDrTok + w + u * (kDrProducers / 32);
            const bool in = pos < a.seq;
            const int64_t tok = tok0 + (in ? pos : 0), gi = tok * a.heads_v + h;
            const T *qp = static_cast<const T *>(a.q) + tok * a.q_stride + int64_t(hk) * a.dk;
            const T *kp = static_cast<const T *>(a.k) + tok * a.k_stride + int64_t(hk) * a.dk;
            const T *vp = static_cast<const T *>(a.v) + tok * a.v_stride + int64_t(h) * a.dv + c0;
#pragma unroll
            for (int j = 0; j < R4; ++j) {
                const int i = lane + 32 * j;
                q[u][j] = in && i < a.dk ? Elem<T>::load(qp + i) : 0.0f;
                k[u][j] = in && i < a.dk ? Elem<T>::load(kp + i) : 0.0f;
            }
            v[u] = in && lane < kDrCols && c0 + lane < a.dv ? Elem<T>::load(vp + lane) : 0.0f;
            g[u] = a.g ? __ldg(a.g + gi) : 0.0f;
            be[u] = a.beta ? __ldg(a.beta + gi) : 1.0f;
            if (a.reset && a.reset[tok])
                g[u] = -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int t = w + u * (kDrProducers / 32);
            float qq = 0.0f, kk = 0.0f, qk = 0.0f;
#pragma unroll
            for (int j = 0; j < R4; ++j) {
                qq = fmaf(q[u][j], q[u][j], qq);
                kk = fmaf(k[u][j], k[u][j], kk);
                qk = fmaf(q[u][j], k[u][j], qk);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                qq += __shfl_xor_sync(0xffffffffu, qq, o);
                kk += __shfl_xor_sync(0xffffffffu, kk, o);
                qk += __shfl_xor_sync(0xffffffffu, qk, o);
            }
            float rq = a.scale, rk = 1.0f;
            if (a.l2norm) {
                rq *= rsqrtf(qq + kDeltaEps);
                rk = rsqrtf(kk + kDeltaEps);
            }
#pragma unroll
            for (int j = 0; j < R4; ++j) {
                buf[Sm::kQ + t * Sm::kDk + lane + 32 * j] = rq * q[u][j];
                buf[Sm::kK + t * Sm::kDk + lane + 32 * j] = rk * k[u][j];
            }
            if (lane < kDrCols)
                buf[Sm::kV + t * kDrCols + lane] = v[u];
            if (lane == 0)
                *reinterpret_cast<float4 *>(buf + Sm::kS + 4 * t) = make_float4(expf(g[u]), be[u], qk * rq * rk, 0.0f);
        }
    };

    const bool consumer = tid < kDrConsumers;
    const int col = tid >> 3, p = tid & 7; // consumer: its column, its lane of 8
    const bool live = consumer && c0 + col < a.dv;
    float S[4 * R4];
#pragma unroll
    for (int i = 0; i < 4 * R4; ++i)
        S[i] = 0.0f;
    const int64_t sbase = bh * a.dk * a.dv + c0 + col;
    if (live && a.h0) {
#pragma unroll
        for (int i = 0; i < 4 * R4; ++i) {
            const int row = 4 * (p + 8 * (i >> 2)) + (i & 3);
            if (row < a.dk)
                S[i] = a.h0[sbase + int64_t(row) * a.dv];
        }
    }
    if (!consumer)
        stage(0, dr_sm);
    __syncthreads();
    T *yp = static_cast<T *>(a.y) + (tok0 * a.heads_v + h) * a.dv + c0 + col;
    const int64_t ystep = int64_t(a.heads_v) * a.dv;
    for (int64_t tile = 0; tile < ntiles; ++tile) {
        if (!consumer) {
            if (tile + 1 < ntiles)
                stage(tile + 1, dr_sm + int((tile + 1) & 1) * Sm::kFloats);
        } else {
            const float *buf = dr_sm + int(tile & 1) * Sm::kFloats;
            const int64_t left = a.seq - tile * kDrTok;
            const int n = left < kDrTok ? int(left) : kDrTok;
            for (int t = 0; t < n; ++t) {
                const float4 *k4 = reinterpret_cast<const float4 *>(buf + Sm::kK + t * Sm::kDk) + p;
                const float4 *q4 = reinterpret_cast<const float4 *>(buf + Sm::kQ + t * Sm::kDk) + p;
                const float4 sc = *reinterpret_cast<const float4 *>(buf + Sm::kS + 4 * t);
                const float v = buf[Sm::kV + t * kDrCols + col];
                if (sc.x == 0.0f) { // a decay of 0 discards the state, whatever it holds
#pragma unroll
                    for (int i = 0; i < 4 * R4; ++i)
                        S[i] = 0.0f;
                }
                float4 k[R4];
                float ks0 = 0.0f, ks1 = 0.0f, qs0 = 0.0f, qs1 = 0.0f;
#pragma unroll
                for (int j = 0; j < R4; ++j) {
                    k[j] = k4[8 * j];
                    const float4 q = q4[8 * j];
                    ks0 = fmaf(k[j].x, S[4 * j], ks0);
                    ks1 = fmaf(k[j].y, S[4 * j + 1], ks1);
                    ks0 = fmaf(k[j].z, S[4 * j + 2], ks0);
                    ks1 = fmaf(k[j].w, S[4 * j + 3], ks1);
                    qs0 = fmaf(q.x, S[4 * j], qs0);
                    qs1 = fmaf(q.y, S[4 * j + 1], qs1);
                    qs0 = fmaf(q.z, S[4 * j + 2], qs0);
                    qs1 = fmaf(q.w, S[4 * j + 3], qs1);
                }
                float ks = ks0 + ks1, qs = qs0 + qs1;
#pragma unroll
                for (int o = 4; o; o >>= 1) {
                    ks += __shfl_xor_sync(0xffffffffu, ks, o);
                    qs += __shfl_xor_sync(0xffffffffu, qs, o);
                }
                const float d = sc.x;
                const float u = sc.y * fmaf(-d, ks, v);
                const float y = fmaf(sc.z, u, d * qs);
#pragma unroll
                for (int j = 0; j < R4; ++j) {
                    const float kv[4] = {k[j].x, k[j].y, k[j].z, k[j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        S[4 * j + e] = fmaf(kv[e], u, d * S[4 * j + e]);
                }
                if (p == 0 && live)
                    Elem<T>::store(yp, y);
                yp += ystep;
            }
        }
        __syncthreads();
    }
    if (live && a.final_state) {
#pragma unroll
        for (int i = 0; i < 4 * R4; ++i) {
            const int row = 4 * (p + 8 * (i >> 2)) + (i & 3);
            if (row < a.dk)
                a.final_state[sbase + int64_t(row) * a.dv] = S[i];
        }
    }
}

// ---- decode step ---------------------------------------------------------------------
//
// Bound by HBM: the state is read and written once, 8 bytes an element.  A CTA owns 32
// columns of one (batch row, head)'s state and holds them in registers between the read
// and the write: thread (r, c) has columns 4 c .. 4 c + 3 of rows r + 16 j, so 8 lanes
// read one 128-byte line, and every state load is issued before the first is used.  The
// partial dot products of the 16 row groups (k . S and q . S for 4 columns; k . k, q . q
// and q . k) are summed by shuffles and once through shared memory; the norms of q and k
// are factors of those sums, so q and k need no pass of their own.

struct DeltaUpdateArgs {
    int64_t batch;
    int heads_k, heads_v, ratio, dk, dv;
    float *state; // [batch, heads_v, dk, dv], updated in place
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride; // elements between consecutive batch rows
    const float *g, *beta;                // [batch, heads_v], nullable
    void *y;                              // [batch, heads_v, dv]
    float scale;
    int l2norm, col_tiles;
};

constexpr int kDuThreads = 128, kDuCols = 32;

// Six CTAs per SM (for dk up to 128) with packed fp32 arithmetic: 162 us for 256 x 32
// states of 128 x 128, the rate of a plain copy; 194 us with scalar arithmetic and four.
// (Tiles of 64 or 128 columns, 171 and 186 us: fewer CTAs whose phases overlap.)
// J: row groups of 16 (dk <= 16 J).  VEC: dv a multiple of 4 and a 16-byte aligned state.
// FULL: dk = 16 J and dv a multiple of 32 as well, so that nothing is guarded (176 us with
// the guards).
template <typename T, int J, bool VEC, bool FULL>
__global__ void __launch_bounds__(kDuThreads, J <= 8 ? 6 : 3) ss_delta_update_kernel(const DeltaUpdateArgs a)
{
    static_assert(VEC || !FULL, "full tiles are read as vectors");
    __shared__ float red[4][8][12];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c4 = tid & 7, r = tid >> 3;
    const int64_t bh = blockIdx.x / unsigned(a.col_tiles);
    const int c = int(blockIdx.x % unsigned(a.col_tiles)) * kDuCols + 4 * c4;
    const int64_t b = bh / a.heads_v;
    const int h = int(bh % a.heads_v), hk = h / a.ratio;
    float *sp = a.state + bh * a.dk * a.dv + c;
    float2 S[J][2]; // columns c, c + 1 and c + 2, c + 3
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int row = r + 16 * j;
        if constexpr (VEC) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (FULL || (row < a.dk && c < a.dv))
                v = __ldcs(reinterpret_cast<const float4 *>(sp + int64_t(row) * a.dv));
            S[j][0] = make_float2(v.x, v.y), S[j][1] = make_float2(v.z, v.w);
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                S[j][e].x = row < a.dk && c + 2 * e < a.dv ? sp[int64_t(row) * a.dv + 2 * e] : 0.0f;
                S[j][e].y = row < a.dk && c + 2 * e + 1 < a.dv ? sp[int64_t(row) * a.dv + 2 * e + 1] : 0.0f;
            }
        }
    }
    const T *qp = static_cast<const T *>(a.q) + b * a.q_stride + int64_t(hk) * a.dk;
    const T *kp = static_cast<const T *>(a.k) + b * a.k_stride + int64_t(hk) * a.dk;
    float k[J];
    float2 ks[2] = {}, qs[2] = {};
    float kk = 0.0f, qq = 0.0f, qdk = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int row = r + 16 * j;
        k[j] = FULL || row < a.dk ? Elem<T>::load(kp + row) : 0.0f;
        const float q = FULL || row < a.dk ? Elem<T>::load(qp + row) : 0.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            ks[e] = __ffma2_rn(make_float2(k[j], k[j]), S[j][e], ks[e]);
            qs[e] = __ffma2_rn(make_float2(q, q), S[j][e], qs[e]);
        }
        kk = fmaf(k[j], k[j], kk);
        qq = fmaf(q, q, qq);
        qdk = fmaf(q, k[j], qdk);
    }
    // k . S and q . S of 4 columns, k . k, q . q, q . k
    float s[11] = {ks[0].x, ks[0].y, ks[1].x, ks[1].y, qs[0].x, qs[0].y, qs[1].x, qs[1].y, kk, qq, qdk};
#pragma unroll
    for (int i = 0; i < 11; ++i) {
        s[i] += __shfl_xor_sync(0xffffffffu, s[i], 8);
        s[i] += __shfl_xor_sync(0xffffffffu, s[i], 16);
    }
    if (lane < 8) {
#pragma unroll
        for (int i = 0; i < 11; ++i)
            red[warp][c4][i] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 11; ++i)
        s[i] = (red[0][c4][i] + red[1][c4][i]) + (red[2][c4][i] + red[3][c4][i]);
    const float rq = a.l2norm ? a.scale * rsqrtf(s[9] + kDeltaEps) : a.scale;
    const float rk = a.l2norm ? rsqrtf(s[8] + kDeltaEps) : 1.0f;
    const int64_t gi = b * a.heads_v + h;
    const float d = a.g ? expf(__ldg(a.g + gi)) : 1.0f;
    const float be = a.beta ? __ldg(a.beta + gi) : 1.0f;
    const float qk = s[10] * rq * rk;
    const T *vp = static_cast<const T *>(a.v) + b * a.v_stride + int64_t(h) * a.dv + c;
    T *yp = static_cast<T *>(a.y) + (b * a.heads_v + h) * a.dv + c;
    if (d == 0.0f) { // a decay of 0 discards the state, whatever it holds
#pragma unroll
        for (int j = 0; j < J; ++j)
            S[j][0] = S[j][1] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[i] = 0.0f;
    }
    float u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float v = FULL || c + e < a.dv ? Elem<T>::load(vp + e) : 0.0f;
        u[e] = be * fmaf(-d * rk, s[e], v);
        if (r == 0 && (FULL || c + e < a.dv))
            Elem<T>::store(yp + e, fmaf(qk, u[e], d * rq * s[4 + e]));
        u[e] *= rk;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int row = r + 16 * j;
        if (!FULL && row >= a.dk)
            break;
        float2 o[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            o[e] = __ffma2_rn(make_float2(k[j], k[j]), make_float2(u[2 * e], u[2 * e + 1]),
                              __fmul2_rn(make_float2(d, d), S[j][e]));
        }
        if constexpr (VEC) {
            if (FULL || c < a.dv)
                __stcs(reinterpret_cast<float4 *>(sp + int64_t(row) * a.dv), make_float4(o[0].x, o[0].y, o[1].x, o[1].y));
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (c + 2 * e < a.dv)
                    sp[int64_t(row) * a.dv + 2 * e] = o[e].x;
                if (c + 2 * e + 1 < a.dv)
                    sp[int64_t(row) * a.dv + 2 * e + 1] = o[e].y;
            }
        }
    }
}

} // namespace ss
