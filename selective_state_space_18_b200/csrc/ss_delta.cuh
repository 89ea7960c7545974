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

// ---- prompt scan in fp32, four tokens a step -----------------------------------------
//
// A CTA owns one (batch row, value head) and 16 or 4 of its value columns: columns of the
// state never meet.  Consumer warps hold the state in registers, a column's dk rows over 8
// or 16 lanes; eight producer warps stage the next 32 tokens, a step of four each, while the
// consumers walk the current ones, and read the tile after that into registers.
//
// What bounds it is the latency of the chain from one state to the next: dot products with
// the state, their sum over the lanes, the write.  So four tokens 0..3 are taken from one
// state S: with a_i their decays, A_i = a_0 .. a_i and D_ij = a_{j+1} .. a_i,
//   u_i = beta_i (v_i - A_i S^T k_i) - sum_{j<i} beta_i D_ij (k_i . k_j) u_j
//   y_i = A_i S^T q_i + sum_{j<=i} D_ij (q_i . k_j) u_j
//   S'  = A_3 S + sum_j D_3j k_j u_j^T
// The factors between tokens come from the producers.  Sums over lanes are exchanges that
// halve the number of values a lane holds: eight values over 8 lanes in 7 shuffles, a
// step's 24 products of rows over a warp in 31.  A step with a decay of 0, or with a
// product of decays past 1e30, is walked token by token: 0 times an infinity or NaN that a
// reset discards, or an infinity times an empty state, would come out of the products.
// All arithmetic is fp32.  It serves fp32 storage, sizes and strides that the tensor-core
// form does not take, and prompts of a few tokens.
//
// Measured (fp32): 2 x 300 tokens x 4 heads of 64: 27.4 us, against 48.7 us one token a
// step; 4 x 2000 tokens x 4 heads of 64: 219 us against 309 us; 300 tokens x 2 heads of 256:
// 44.5 us against 86 us.  What has a few tokens only, or many heads on every SM, loses a
// little (16 heads of 128 x 4 tokens 5.6 us against 4.7; 256 heads x 300 tokens 669 us
// against 634).

// LN: lanes a column.  8 with 16 columns a CTA (four consumer warps), or 16 with 4 columns
// (two).  A consumer warp issues an instruction in about five cycles, so a step lasts as long
// as its instructions: 16 lanes halve those of the products, for one more exchange in the
// sums; and 16-byte reads that the columns of a warp share take four turns of the SM's path to
// shared memory, which fewer warps crowd less.  Where the grid is small, the narrow form also
// spreads over more SMs.
constexpr int kDrTok = 32, kDrStep = 4, kDrProducers = 256;
constexpr int dr_cols(int ln) { return ln == 8 ? 16 : 4; }
constexpr int dr_threads(int ln) { return dr_cols(ln) * ln + kDrProducers; }

template <int R4, int LN> struct DeltaRecSmem { // floats of one staging buffer
    static constexpr int kDk = 32 * R4; // padded key size
    static constexpr int kVRow = kDrTok + 4;
    static constexpr int kK = 0, kQ = kDrTok * kDk, kV = 2 * kDrTok * kDk /* [column][token] */, kS = kV + dr_cols(LN) * kVRow;
    // factors of a step: A_i, beta_i, D_3j, a_i (4 each), beta_i D_ij k_i.k_j for ij = 10 20 21 30
    // 31 32, whether it goes token by token, (unused), D_ij q_i.k_j as 4 x 4 rows
    static constexpr int kA = 0, kBeta = 4, kD3 = 8, kDecay = 12, kC = 16, kSingle = 22, kE = 24, kStep = 40;
    static constexpr int kFloats = kS + kStep * (kDrTok / kDrStep);
    static constexpr size_t kBytes = 2 * size_t(kFloats) * 4;
};

// Sums of N values over groups of N lanes, `step` apart: lane l of a group is left with that
// of value l.
template <int N> __device__ __forceinline__ float dr_sums(float (&v)[N], int lane, int step = 1)
{
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o * step);
        }
    }
    return v[0];
}

template <typename T, int R4, int LN>
__global__ void __launch_bounds__(dr_threads(LN)) ss_delta_rec_kernel(const DeltaArgs a)
{
    using Sm = DeltaRecSmem<R4, LN>;
    constexpr int RJ = 8 * R4 / LN; // groups of four rows a lane
    static_assert(RJ * LN == 8 * R4, "the padded key size divides among the lanes");
    constexpr int kDrCols = dr_cols(LN), kDrConsumers = kDrCols * LN;
    constexpr int kVs = (kDrStep * kDrCols + 31) / 32; // values of v a producer lane loads
    extern __shared__ __align__(16) float dr_sm[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int tiles = (a.dv + kDrCols - 1) / kDrCols;
    const int c0 = int(blockIdx.x % unsigned(tiles)) * kDrCols;
    const int64_t bh = blockIdx.x / unsigned(tiles);
    const int64_t b = bh / a.heads_v;
    const int h = int(bh % a.heads_v), hk = h / a.ratio;
    const int64_t tok0 = b * a.seq; // first token of this batch row
    const int64_t ntiles = (a.seq + kDrTok - 1) / kDrTok;

    if (tid >= kDrConsumers) {
        // ======================= producers: warp w has step w of every tile ================
        const int w = (tid - kDrConsumers) >> 5;
        float k[4][R4], q[4][R4], v[kVs], g, be;
        // Tokens past the end are staged as k = q = v = 0, beta = 0, no decay: they change nothing.
        auto fetch = [&](int64_t tile) {
            const int64_t pos0 = tile * kDrTok + kDrStep * w;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool in = pos0 + u < a.seq;
                const int64_t tok = tok0 + (in ? pos0 + u : 0);
                const T *qp = static_cast<const T *>(a.q) + tok * a.q_stride + int64_t(hk) * a.dk;
                const T *kp = static_cast<const T *>(a.k) + tok * a.k_stride + int64_t(hk) * a.dk;
#pragma unroll
                for (int j = 0; j < R4; ++j) {
                    const int i = lane + 32 * j;
                    k[u][j] = in && i < a.dk ? Elem<T>::load(kp + i) : 0.0f;
                    q[u][j] = in && i < a.dk ? Elem<T>::load(qp + i) : 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < kVs; ++u) { // 4 tokens x kDrCols columns
                const int64_t pos = pos0 + (32 * u + lane) / kDrCols;
                const int c = c0 + lane % kDrCols;
                v[u] = 32 * u + lane < kDrStep * kDrCols && pos < a.seq && c < a.dv
                           ? Elem<T>::load(static_cast<const T *>(a.v) + (tok0 + pos) * a.v_stride + int64_t(h) * a.dv + c)
                           : 0.0f;
            }
            g = 0.0f, be = 0.0f; // lane u < 4: of token u
            if (lane < 4 && pos0 + lane < a.seq) {
                const int64_t tok = tok0 + pos0 + lane, gi = tok * a.heads_v + h;
                g = a.g ? __ldg(a.g + gi) : 0.0f;
                be = a.beta ? __ldg(a.beta + gi) : 1.0f;
                if (a.reset && a.reset[tok])
                    g = -INFINITY;
            }
        };
        auto stage = [&](float *buf) {
            float *f = buf + Sm::kS + Sm::kStep * w;
            // value 4 i + j (j <= i): q_i . k_j; 16 + 4 i + j: k_i . k_j; 17, 18, 19, 22: |q_i|^2
            float s[32] = {};
#pragma unroll
            for (int x = 0; x < R4; ++x) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int j = 0; j <= i; ++j) {
                        s[4 * i + j] = fmaf(q[i][x], k[j][x], s[4 * i + j]);
                        s[16 + 4 * i + j] = fmaf(k[i][x], k[j][x], s[16 + 4 * i + j]);
                    }
                    const int qi = i < 3 ? 17 + i : 22;
                    s[qi] = fmaf(q[i][x], q[i][x], s[qi]);
                }
            }
            const float sum = dr_sums<32>(s, lane);
            const float r = a.l2norm ? rsqrtf(sum + kDeltaEps) : 1.0f;
            float rk[4], rq[4], dec[4], beta[4];
            const float e = expf(g);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                rk[u] = __shfl_sync(0xffffffffu, r, 16 + 5 * u);
                rq[u] = a.scale * __shfl_sync(0xffffffffu, r, u < 3 ? 17 + u : 22);
                dec[u] = __shfl_sync(0xffffffffu, e, u);
                beta[u] = __shfl_sync(0xffffffffu, be, u);
#pragma unroll
                for (int j = 0; j < R4; ++j) {
                    buf[Sm::kK + (kDrStep * w + u) * Sm::kDk + lane + 32 * j] = rk[u] * k[u][j];
                    buf[Sm::kQ + (kDrStep * w + u) * Sm::kDk + lane + 32 * j] = rq[u] * q[u][j];
                }
            }
#pragma unroll
            for (int u = 0; u < kVs; ++u)
                if (32 * u + lane < kDrStep * kDrCols)
                    buf[Sm::kV + lane % kDrCols * Sm::kVRow + kDrStep * w + (32 * u + lane) / kDrCols] = v[u];
            // this lane's product: factors picked by its i and j
            const int i = (lane >> 2) & 3, j = lane & 3;
            auto pick = [](const float (&x)[4], int n) { return n < 2 ? (n ? x[1] : x[0]) : (n == 2 ? x[2] : x[3]); };
            const float d = (j < 1 && i >= 1 ? dec[1] : 1.0f) * (j < 2 && i >= 2 ? dec[2] : 1.0f) * (j < 3 && i >= 3 ? dec[3] : 1.0f);
            const float dk = d * (sum * pick(rk, j));
            if (lane < 16)
                f[Sm::kE + lane] = j <= i ? dk * pick(rq, i) : 0.0f;
            else if (j < i)
                f[Sm::kC + i * (i - 1) / 2 + j] = pick(beta, i) * (dk * pick(rk, i));
            const float a01 = dec[0] * dec[1], a12 = dec[1] * dec[2], a23 = dec[2] * dec[3];
            if (lane == 0) {
                const float4 A = make_float4(dec[0], a01, a01 * dec[2], a01 * a23);
                const float4 D = make_float4(a12 * dec[3], a23, dec[3], 1.0f);
                *reinterpret_cast<float4 *>(f + Sm::kA) = A;
                *reinterpret_cast<float4 *>(f + Sm::kBeta) = make_float4(beta[0], beta[1], beta[2], beta[3]);
                *reinterpret_cast<float4 *>(f + Sm::kD3) = D;
                *reinterpret_cast<float4 *>(f + Sm::kDecay) = make_float4(dec[0], dec[1], dec[2], dec[3]);
                const float most = fmaxf(fmaxf(fmaxf(A.x, A.y), fmaxf(A.z, A.w)),
                                         fmaxf(fmaxf(fmaxf(D.x, D.y), fmaxf(D.z, a12)), fmaxf(dec[1], dec[2])));
                const bool zero = dec[0] == 0.0f || dec[1] == 0.0f || dec[2] == 0.0f || dec[3] == 0.0f;
                f[Sm::kSingle] = zero || most > 1e30f ? 1.0f : 0.0f;
            }
        };
        fetch(0);
        stage(dr_sm);
        __syncthreads();
        if (ntiles > 1)
            fetch(1);
        for (int64_t tile = 0; tile < ntiles; ++tile) {
            if (tile + 1 < ntiles) {
                stage(dr_sm + int((tile + 1) & 1) * Sm::kFloats);
                if (tile + 2 < ntiles)
                    fetch(tile + 2);
            }
            __syncthreads();
        }
        return;
    }

    // ======================= consumers: LN lanes a column ==================================
    const int col = tid / LN, p = tid % LN;
    const bool live = c0 + col < a.dv;
    float2 S[2 * RJ]; // rows 4 (p + LN j) .. + 3
    const int64_t sbase = bh * a.dk * a.dv + c0 + col;
#pragma unroll
    for (int i = 0; i < 2 * RJ; ++i) {
        const int row = 4 * (p + LN * (i >> 1)) + 2 * (i & 1);
        const bool in = live && a.h0;
        S[i].x = in && row < a.dk ? a.h0[sbase + int64_t(row) * a.dv] : 0.0f;
        S[i].y = in && row + 1 < a.dk ? a.h0[sbase + int64_t(row + 1) * a.dv] : 0.0f;
    }
    __syncthreads();
    const int64_t ystep = int64_t(a.heads_v) * a.dv;
    // of the eight sums of a step the lane is left with number `mine`: S^T k of token yi, or
    // from 4 on S^T q of it, whose output the (first) lane writes
    constexpr int kSame = LN / 8;
    const int mine = p / kSame, yi = mine & 3;
    const bool writes = live && mine >= 4 && p % kSame == 0;
    T *yp = static_cast<T *>(a.y) + ((tok0 + yi) * a.heads_v + h) * a.dv + c0 + col;
    for (int64_t tile = 0; tile < ntiles; ++tile) {
        const float *buf = dr_sm + int(tile & 1) * Sm::kFloats;
        const int64_t left = a.seq - tile * kDrTok;
        const int n = left < kDrTok ? int(left) : kDrTok;
#pragma unroll 1
        for (int t = 0; t < n; t += kDrStep, yp += kDrStep * ystep) {
            const float4 *k4 = reinterpret_cast<const float4 *>(buf + Sm::kK + t * Sm::kDk) + p;
            const float4 *q4 = reinterpret_cast<const float4 *>(buf + Sm::kQ + t * Sm::kDk) + p;
            const float *f = buf + Sm::kS + Sm::kStep * (t / kDrStep), *vp = buf + Sm::kV + col * Sm::kVRow + t;
            if (f[Sm::kSingle] != 0.0f) { // token by token
#pragma unroll 1
                for (int u = 0; u < 4; ++u) {
                    const float d = f[Sm::kDecay + u];
                    float2 ks2 = make_float2(0.0f, 0.0f), qs2 = ks2;
#pragma unroll
                    for (int i = 0; i < 2 * RJ; ++i) // a decay of 0 discards the state, whatever it holds
                        S[i] = d == 0.0f ? make_float2(0.0f, 0.0f) : __fmul2_rn(make_float2(d, d), S[i]);
#pragma unroll
                    for (int j = 0; j < RJ; ++j) {
                        const float4 kv = k4[u * (Sm::kDk / 4) + LN * j], qv = q4[u * (Sm::kDk / 4) + LN * j];
                        ks2 = __ffma2_rn(make_float2(kv.x, kv.y), S[2 * j], ks2);
                        qs2 = __ffma2_rn(make_float2(qv.x, qv.y), S[2 * j], qs2);
                        ks2 = __ffma2_rn(make_float2(kv.z, kv.w), S[2 * j + 1], ks2);
                        qs2 = __ffma2_rn(make_float2(qv.z, qv.w), S[2 * j + 1], qs2);
                    }
                    float ks = ks2.x + ks2.y, qs = qs2.x + qs2.y;
#pragma unroll
                    for (int o = LN / 2; o; o >>= 1) {
                        ks += __shfl_xor_sync(0xffffffffu, ks, o);
                        qs += __shfl_xor_sync(0xffffffffu, qs, o);
                    }
                    const float x = f[Sm::kBeta + u] * (vp[u] - ks);
                    if (writes && yi == u && t + u < n)
                        Elem<T>::store(yp, fmaf(f[Sm::kE + 5 * u], x, qs));
#pragma unroll
                    for (int j = 0; j < RJ; ++j) {
                        const float4 kv = k4[u * (Sm::kDk / 4) + LN * j];
                        S[2 * j] = __ffma2_rn(make_float2(kv.x, kv.y), make_float2(x, x), S[2 * j]);
                        S[2 * j + 1] = __ffma2_rn(make_float2(kv.z, kv.w), make_float2(x, x), S[2 * j + 1]);
                    }
                }
                continue;
            }
            float2 s2[8] = {}; // S^T k of the four tokens, S^T q of them
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 kv = k4[u * (Sm::kDk / 4) + LN * j], qv = q4[u * (Sm::kDk / 4) + LN * j];
                    s2[u] = __ffma2_rn(make_float2(kv.x, kv.y), S[2 * j], s2[u]);
                    s2[4 + u] = __ffma2_rn(make_float2(qv.x, qv.y), S[2 * j], s2[4 + u]);
                    s2[u] = __ffma2_rn(make_float2(kv.z, kv.w), S[2 * j + 1], s2[u]);
                    s2[4 + u] = __ffma2_rn(make_float2(qv.z, qv.w), S[2 * j + 1], s2[4 + u]);
                }
            }
            // A_i S^T k_i and what token i writes by itself, or A_i S^T q_i
            const float4 D = *reinterpret_cast<const float4 *>(f + Sm::kD3), E = *reinterpret_cast<const float4 *>(f + Sm::kE + 4 * yi);
            const float4 ca = *reinterpret_cast<const float4 *>(f + Sm::kC);
            const float2 cb = *reinterpret_cast<const float2 *>(f + Sm::kC + 4);
            const float A3 = f[Sm::kA + 3], Ai = f[Sm::kA + yi], bi = f[Sm::kBeta + yi], vi = vp[yi];
            float s[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                s[u] = s2[u].x + s2[u].y;
            float sum = dr_sums<8>(s, p / kSame, kSame);
            if (LN == 16)
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            const float as = Ai * sum;
            const float own = bi * (vi - as);
            const float u0 = __shfl_sync(0xffffffffu, own, 0, LN);
            const float x1 = __shfl_sync(0xffffffffu, own, kSame, LN), x2 = __shfl_sync(0xffffffffu, own, 2 * kSame, LN),
                        x3 = __shfl_sync(0xffffffffu, own, 3 * kSame, LN);
            const float u1 = fmaf(-ca.x, u0, x1);
            const float u2 = fmaf(-ca.z, u1, fmaf(-ca.y, u0, x2));
            const float u3 = fmaf(-cb.y, u2, fmaf(-cb.x, u1, fmaf(-ca.w, u0, x3)));
            const float w[4] = {D.x * u0, D.y * u1, D.z * u2, u3};
#pragma unroll
            for (int i = 0; i < 2 * RJ; ++i)
                S[i] = __fmul2_rn(make_float2(A3, A3), S[i]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int j = 0; j < RJ; ++j) {
                    const float4 kv = k4[u * (Sm::kDk / 4) + LN * j];
                    S[2 * j] = __ffma2_rn(make_float2(kv.x, kv.y), make_float2(w[u], w[u]), S[2 * j]);
                    S[2 * j + 1] = __ffma2_rn(make_float2(kv.z, kv.w), make_float2(w[u], w[u]), S[2 * j + 1]);
                }
            }
            float y = fmaf(E.x, u0, as); // later tokens' u may be infinite or NaN
            y = yi >= 1 ? fmaf(E.y, u1, y) : y;
            y = yi >= 2 ? fmaf(E.z, u2, y) : y;
            y = yi >= 3 ? fmaf(E.w, u3, y) : y;
            if (writes && t + yi < n)
                Elem<T>::store(yp, y);
        }
        __syncthreads();
    }
    if (live && a.final_state) {
#pragma unroll
        for (int i = 0; i < 2 * RJ; ++i) {
            const int row = 4 * (p + LN * (i >> 1)) + 2 * (i & 1);
            if (row < a.dk)
                a.final_state[sbase + int64_t(row) * a.dv] = S[i].x;
            if (row + 1 < a.dk)
                a.final_state[sbase + int64_t(row + 1) * a.dv] = S[i].y;
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

// Six CTAs per SM (for dk up to 128) with packed fp32 arithmetic: 162-168 us for 256 x 32
// states of 128 x 128 (1.07 GB moved) alone, two states in turn, the rate of a plain copy, and
// 187 us in a run over three states, 88% of it; alone 194 us with scalar arithmetic and four.
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
