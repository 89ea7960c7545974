// ss_delta_tc.cuh -- the gated delta rule's prompt scan in chunked form on the tensor
// cores: a kernel that prepares every chunk by itself, and a kernel that walks the chunks.
//
// With the entering state H [dk x dv] and, inside a chunk of 64 tokens (i, j = 0..63),
//   D_ij = exp(g_{j+1} + ... + g_i)   (0 when a reset lies in j+1..i, or j > i)
//   E_i  = the same from the chunk's start to i, F_j = D_63,j
//   r_i, p_i = 1 / |k_i| and scale / |q_i|  (1 and scale without the norm)
// the recurrence S_t = a_t S_{t-1} + k_t u_t^T, u_t = beta_t (v_t - a_t S_{t-1}^T k_t)
// unrolls to a triangular system for the writes u and three products:
//   (I + A) U = diag(beta) (V - diag(c) K H),  A_ij = beta_i r_i r_j D_ij k_i.k_j (j < i),
//                                              c_i = r_i E_i
//   Y  = diag(s) Q H + P U,    s_i = p_i E_i, P_ij = p_i r_j D_ij q_i.k_j (j <= i)
//   H' = E_63 H + K^T diag(w) U,               w_j = r_j F_j
// The norms of q and k are factors of rows and columns, so q and k enter every product as
// they are stored.
//
// The preparation (ss_delta_prep_kernel, one CTA per chunk and value head) needs no state:
// K K^T and Q K^T, the decays, T = (I + A)^{-1} diag(beta) by substitution in fp32, and
// per chunk and value head a 25 KB block of the workspace: T and P (each split into a bf16
// high part and a bf16 remainder) as operand tiles, c, w, s and E_63.
//
// The walk (ss_delta_walk_kernel, one CTA per head and 128 value columns) keeps H in fp32
// registers, transposed: tensor-memory lane = value column.  Every product then takes its
// left operand from tensor memory, where the element-wise steps leave it with no pass
// through shared memory, and its right operand straight from the TMA tiles of k and q:
//   KH^T [128 x 64]  = H^T K^T              R^T = V^T - KH^T diag(c)
//   U^T  [128 x 64]  = R^T T^T              (only the blocks of T on and below the diagonal)
//   Y^T  [128 x 64]  = (H^T Q^T + (w o U)^T P'^T) diag(s),   P'_ij = q_i.k_j / E_63  (j <= i)
//   dH^T [128 x dk]  = (w o U)^T K          H = E_63 H + dH
// since P_ij = s_i P'_ij w_j without a cut in the chunk.  One operand serves both products.
// P' and w are only in range where the chunk's decays are.  With a cut in the chunk, or decays
// beyond 2^-60 in all, s and w are taken apart into powers of two and the rest, from 1 to 2:
// the walk scales the rows of Q and K by the powers in shared memory, which rounds nothing, the
// rest takes the place of s and w, and P'_ij is P_ij over both (the block says which).
//
// Few heads and a long prompt leave most SMs without a walk.  The sequence is then cut into
// segments that are walked at once, in two passes ("s6_reset" blog draft, Associative
// Boundary Resetting, for matrix states): a segment acts on the state that enters it as
// S -> M S + N, so pass 1 walks every segment but the last for N, its end state from zero
// (the first from h0), and every one but the first and the last for M, its end state from
// the identity with v = 0; ss_delta_join_kernel chains them in fp32, and pass 2 walks every
// segment from its entering state with outputs.  A segment whose decays underflow has an M
// of exactly 0: its walk ends there, and the join has nothing to multiply.
//
// Precision.  q, k and v are bf16 inputs and enter exactly.  On the way from state to
// state the computed operands (H, R, T, w o U) are split, x = hi + lo to 2^-17, and their
// products summed in fp32, so the final state follows fp32 arithmetic to about 5e-6 of
// its size.  So do those on the way to the outputs (H, w o U, P'): where keys resemble each
// other the terms of P U are many times its sum, and operands of 8 bits were off by up to 0.13
// in outputs of order one.  Output error 1.7e-3 of the norm, which is the rounding of the output
// itself.
//
// Decays.  The cumulative log2 decays are kept as a part of multiples of 1/64, which sums
// and differences exactly, and a remainder below 1/128 a token, each with an exponential of its
// own, so the factors from the chunk's start or to its end are right to 7e-7 however much the
// chunk decays in all (1.7e-6 over 2^-53 with one exponential of the sum, and worse with the
// roundings of g log2(e) added up).  A token whose decay is
// zero in fp32 (a reset, -inf, below 2^-160) cuts: cut counts tell which pairs it parts.
// A cut at a chunk's first token leaves the chunk itself alone: the chunk before it hands
// on a state of zero (and h0 is not read).  A sequence without h0 begins the same way, so
// within a segment a document that starts a chunk gives the same bits as on its own.
#pragma once

#include <cuda.h>
#include "ss_device.cuh"
#include "ss_gated_tc.cuh" // tensor-memory and tcgen05 primitives
#include "ss_state_update.cuh" // bulk_load
#include "ss_sync.cuh"
#include "ss_delta.cuh"

namespace ss {

constexpr int kDcChunk = 64; // tokens per chunk
constexpr float kDcLog2eRest = float(1.4426950408889634 - double(kLog2e)); // log2(e) beyond kLog2e

// A block: T hi, T lo, four arrays of 64 floats (c, w, s; then E_63, the mode: 0, or 1 for cuts
// and strong decays, and from kDcPow on the powers of two of w and of s as the exponents' eight
// bits), then P' hi, P' lo.  A matrix is
// four slices ks of 32-byte rows in the 32-byte swizzle: columns 16 ks .. 16 ks + 15, rows
// 0..63 of the first two slices and 32..63 of the last two (the rest is above the diagonal
// and 0).  Products with it accumulate into two halves of 32 tokens each, always with
// N = 32: MMAs into one accumulator are only ordered among themselves when they have one
// shape.
constexpr int kDcMat = 6144;
__host__ __device__ constexpr int dc_slice(int ks) { return ks < 2 ? 2048 * ks : 4096 + 1024 * (ks - 2); }
constexpr int kDcThi = 0, kDcTlo = kDcMat, kDcC = 2 * kDcMat, kDcW = kDcC + 256, kDcS = kDcW + 256, kDcE = kDcS + 256,
              kDcP = kDcE + 256;
constexpr int kDcHead = kDcP;                     // the part loaded ahead of P
constexpr int kDcBlockBytes = kDcP + 2 * kDcMat;  // workspace per chunk and value head
constexpr int kDcPow = kDcE + 16;
static_assert(kDcHead % 1024 == 0 && kDcBlockBytes == 25600, "workspace block");

// x = m 2^e: the bits of the power of two (0 for 0 and below float32's normal range) and m (1 to
// 2 in size, with the sign), whose product is x, or 0 there.
__device__ __forceinline__ unsigned char dc_power(float x) { return (unsigned char)(__float_as_uint(x) >> 23); }
__device__ __forceinline__ float dc_mantissa(float s)
{
    return __uint_as_float((__float_as_uint(s) & 0x807fffffu) | 0x3f800000u);
}

// Byte offset of element (i, j) of a matrix in its slices (i >= 32 when j >= 32): the
// 16-byte half of a 32-byte row is XORed with bit 2 of the row (address bit 4 with bit 7).
__device__ __forceinline__ int dc_elem(int i, int j)
{
    const int r = i - (j & 32), o = (j & 15) * 2;
    return dc_slice(j >> 4) + r * 32 + (o ^ ((r & 4) << 2));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t saddr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr));
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether the state is discarded before token `tok` (an index over all batch rows).
__device__ __forceinline__ bool dc_cut(const uint8_t *reset, const float *g, int64_t tok, int heads_v, int h)
{
    return (reset && reset[tok]) || (g && __ldg(g + tok * heads_v + h) * kLog2e < -160.0f);
}

// 16 bytes global -> shared memory, or zeros.
__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}

struct DeltaPrepArgs {
    DeltaArgs d;
    int nchunks;
    unsigned char *blocks; // [batch, heads_v, nchunks] blocks
};

// ---- preparation ---------------------------------------------------------------------
//
// 128 threads, five CTAs per SM.  Warp w owns rows 16 w .. 16 w + 15: it computes them of
// K K^T and Q K^T with mma.sync, up to the diagonal (64 x 64 products of a microsecond in
// all do not repay tensor-memory round trips), scales them by the decays into A, which
// stays in its registers as fragments, and P, and builds its rows of T = (I + A)^{-1} block
// by block: the inverse T_ww of its 16 x 16 diagonal block by substitution, one column a
// lane, and then, j = w - 1 down to 0,
//   T_wj = -T_ww W,   W = sum_{j <= k < w} A_wk T_kj
// with mma.sync on tf32 operands split in two (22 bits), which keeps the error of fp32
// arithmetic.  A product's result fragment is the left operand of the next one as it
// stands, and the transpose of its right operand (the keys of a step taken in the order
// 0, 2, 4, 6, 1, 3, 5, 7 on both sides), so W is computed as W^T = sum T_kj^T A_wk^T, and
// only the T_kj^T pass from warp to warp, through shared memory.  (Value heads that share a
// key head repeat its two products, a tenth of the work: kept in registers over the heads
// they cost the occupancy that hides the rest.)
//
// Measured: 135 us for 8192 chunks of 128 keys (8 x 2048 tokens x 32 heads), 145 us where an
// eighth of the heads decays strongly; 139 MB read and 157 MB written, 2.0 TB/s: HBM does not
// bound it.  8600 warp instructions a chunk, issued in 47% of the cycles by 19 warps an SM:
// instruction issue and the latencies between them.  With P in one part (136 us on the same
// inputs as 145), steps left out in turn: the merges of T 33 us, K K^T and Q K^T 31 us, A and P
// 18 us, the block's store 8 us; without any of the work 32 us; and with T built by packed fp32
// arithmetic on A in shared memory 150 us.

constexpr int kDpThreads = 128;
constexpr int kDpRow = 136;   // elements between rows of the q and k tiles (272 bytes)
constexpr int kDpDRow = 20;   // floats between rows of a diagonal block
struct DeltaPrepSmem {        // the image, T_kj^T and the diagonal blocks take the place of the tiles
    static constexpr int kK = 0, kQ = kDcChunk * kDpRow * 2;
    static constexpr int kImg = 0;                    // T hi, T lo, P' hi, P' lo
    static constexpr int kTT = kImg + 4 * kDcMat;     // T_kj^T, k < 3, as fragments: [6 blocks][32 lanes][8]
    static constexpr int kDiag = kTT + 6 * 1024;      // [4 warps][16][kDpDRow]
    static constexpr int kScal = 2 * kQ + 1024; // per token: Gh, Gl, cut count, r, p, beta, r / E, beta r E (64 floats each)
    static constexpr int kBytes = kScal + 8 * 256 + 16;
    static_assert(kDiag + 4 * 16 * kDpDRow * 4 <= kScal, "inside the tiles");
};

// A 16 x 16 block as the result fragment of two m16n8 products: f[4 n + 2 x + e] is row
// t / 4 + 8 x, column 8 n + 2 (t % 4) + e.
struct DpFrag {
    float f[8];
};

__device__ __forceinline__ void mma_1688_tf32(float *d, const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A block as an operand: the first 11 bits of each element and the rest.
struct DpOp {
    uint32_t h[8], l[8];
};
__device__ __forceinline__ DpOp dp_split(const DpFrag &m)
{
    DpOp o;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        o.h[i] = __float_as_uint(m.f[i]) & 0xffffe000u;
        o.l[i] = __float_as_uint(m.f[i] - __uint_as_float(o.h[i]));
    }
    return o;
}

// d += m n, with n given as its transpose.
__device__ __forceinline__ void dp_mul(DpFrag &d, const DpOp &m, const DpOp &nt)
{
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        const uint32_t ah[4] = {m.h[4 * ks], m.h[4 * ks + 2], m.h[4 * ks + 1], m.h[4 * ks + 3]};
        const uint32_t al[4] = {m.l[4 * ks], m.l[4 * ks + 2], m.l[4 * ks + 1], m.l[4 * ks + 3]};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int i = 4 * ks + 2 * n;
            mma_1688_tf32(d.f + 4 * n, al, nt.h[i], nt.h[i + 1]);
            mma_1688_tf32(d.f + 4 * n, ah, nt.l[i], nt.l[i + 1]);
            mma_1688_tf32(d.f + 4 * n, ah, nt.h[i], nt.h[i + 1]);
        }
    }
}

// A block of packed pairs (rows 16 i, columns 16 j of a matrix) into its slice of the
// image: matrix lane / 8 of the four 8 x 8, row lane % 8.
__device__ __forceinline__ void dp_store_block(uint32_t mat, int i, int j, int lane, const uint32_t (&w)[4])
{
    const int row = 16 * i + 8 * ((lane >> 3) & 1) + (lane & 7);
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     mat + uint32_t(dc_elem(row, 16 * j + 8 * (lane >> 4)))),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}

__global__ void __launch_bounds__(kDpThreads, 5) ss_delta_prep_kernel(const DeltaPrepArgs a)
{
    using Sm = DeltaPrepSmem;
    extern __shared__ __align__(128) unsigned char dp_sm[];
    const DeltaArgs &d = a.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = int(blockIdx.x % unsigned(d.heads_v)), hk = h / d.ratio;
    const int64_t bc = blockIdx.x / unsigned(d.heads_v);
    const int chunk = int(bc % a.nchunks);
    const int64_t b = bc / a.nchunks;
    const int64_t t0 = int64_t(chunk) * kDcChunk, tok0 = b * d.seq + t0;
    const int n = int(d.seq - t0 < kDcChunk ? d.seq - t0 : kDcChunk); // tokens of this chunk
    __nv_bfloat16 *sk = reinterpret_cast<__nv_bfloat16 *>(dp_sm + Sm::kK);
    __nv_bfloat16 *sq = reinterpret_cast<__nv_bfloat16 *>(dp_sm + Sm::kQ);
    const uint32_t img = smem_u32(dp_sm + Sm::kImg);
    float *sGh = reinterpret_cast<float *>(dp_sm + Sm::kScal), *sGl = sGh + 64, *sR = sGh + 192, *sP = sGh + 256,
          *sBeta = sGh + 320, *sF = sGh + 384, *sB = sGh + 448;
    int *sN = reinterpret_cast<int *>(sGh + 128);
    float *sRed = sGh + 512; // the first warp's totals

    // q and k rows, zero beyond dk and beyond the sequence
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(d.k) + tok0 * d.k_stride + int64_t(hk) * d.dk;
    const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(d.q) + tok0 * d.q_stride + int64_t(hk) * d.dk;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = tid + kDpThreads * i, r = e >> 4, c = (e & 15) * 8;
        const bool in = r < n && c < d.dk;
        cp_async16(sk + r * kDpRow + c, in ? kp + r * d.k_stride + c : kp, in);
        cp_async16(sq + r * kDpRow + c, in ? qp + r * d.q_stride + c : qp, in);
    }
    // ---- decays: thread t < 64 has token t -----------------------------------------------
    float gh = 0.0f, gl = 0.0f, be = 0.0f;
    int cut = 0;
    if (tid < 64) {
        if (tid < n) {
            const int64_t gi = (tok0 + tid) * d.heads_v + h;
            be = d.beta ? __ldg(d.beta + gi) : 1.0f;
            const float g = d.g ? __ldg(d.g + gi) : 0.0f, g2 = g * kLog2e;
            if ((d.reset && d.reset[tok0 + tid]) || g2 < -160.0f) {
                cut = tid > 0; // (at the first token: see above)
            } else if (tid > 0 || chunk > 0 || d.h0 || g2 != g2) { // (an empty state has nothing to lose)
                gh = rintf(g2 * 64.0f) * (1.0f / 64.0f);
                // (g log2(e) - gh, without the roundings of the product and of log2(e))
                gl = fmaf(g, kDcLog2eRest, fmaf(g, kLog2e, -gh));
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float uh = __shfl_up_sync(0xffffffffu, gh, o), ul = __shfl_up_sync(0xffffffffu, gl, o);
            const int uc = __shfl_up_sync(0xffffffffu, cut, o);
            if (lane >= o) {
                gh += uh;
                gl += ul;
                cut += uc;
            }
        }
        if (tid == 31) {
            sRed[0] = gh;
            sRed[1] = gl;
            sRed[2] = __int_as_float(cut);
        }
        if (tid == 0)
            sRed[3] = t0 + kDcChunk < d.seq && dc_cut(d.reset, d.g, tok0 + kDcChunk, d.heads_v, h) ? 0.0f : 1.0f;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // this warp's 16 rows of K K^T and Q K^T, columns 0 .. 16 warp + 15, and the 16 x 16
    // diagonal block of Q Q^T (for the lengths)
    float kk[8][4], qk[8][4], qq[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            kk[i][e] = qk[i][e] = qq[i & 1][e] = 0.0f;
    {
        const uint32_t kb = smem_u32(sk), qb = smem_u32(sq);
        // A fragments: rows 16 warp + lane % 16, columns 8 (lane / 16); B fragments (two
        // n-tiles): token rows (lane % 8) + 8 (lane / 16), columns 8 ((lane / 8) % 2)
        const uint32_t ao = uint32_t((16 * warp + (lane & 15)) * kDpRow + 8 * (lane >> 4)) * 2;
        const uint32_t bo = uint32_t(((lane & 7) + 8 * (lane >> 4)) * kDpRow + 8 * ((lane >> 3) & 1)) * 2;
        const int nks = (d.dk + 15) / 16;
#pragma unroll 2
        for (int ks = 0; ks < nks; ++ks) {
            uint32_t ak[4], aq[4], bq[4];
            ldmatrix_x4(ak, kb + ao + 32 * ks);
            ldmatrix_x4(aq, qb + ao + 32 * ks);
            ldmatrix_x4(bq, qb + bo + uint32_t(16 * warp * kDpRow) * 2 + 32 * ks);
            mma_16816(qq[0], aq, bq[0], bq[1]);
            mma_16816(qq[1], aq, bq[2], bq[3]);
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                if (np <= warp) {
                    uint32_t bk[4];
                    ldmatrix_x4(bk, kb + bo + uint32_t(16 * np * kDpRow) * 2 + 32 * ks);
                    mma_16816(kk[2 * np], ak, bk[0], bk[1]);
                    mma_16816(kk[2 * np + 1], ak, bk[2], bk[3]);
                    mma_16816(qk[2 * np], aq, bk[0], bk[1]);
                    mma_16816(qk[2 * np + 1], aq, bk[2], bk[3]);
                }
            }
        }
    }
    // lengths, from the diagonals: row t / 4 (+ 8 in the second tile) is in the thread
    // whose column pair 2 (t % 4) holds it
    {
        const int g = lane >> 2, t2 = 2 * (lane & 3);
        if (g == t2 || g == t2 + 1) {
            const int e = g - t2;
            float k0 = 0.0f, k1 = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w == warp) {
                    k0 = e ? kk[2 * w][1] : kk[2 * w][0];
                    k1 = e ? kk[2 * w + 1][3] : kk[2 * w + 1][2];
                }
            }
            const float q0 = e ? qq[0][1] : qq[0][0], q1 = e ? qq[1][3] : qq[1][2];
            sR[16 * warp + g] = d.l2norm ? rsqrtf(k0 + kDeltaEps) : 1.0f;
            sR[16 * warp + g + 8] = d.l2norm ? rsqrtf(k1 + kDeltaEps) : 1.0f;
            sP[16 * warp + g] = d.l2norm ? d.scale * rsqrtf(q0 + kDeltaEps) : d.scale;
            sP[16 * warp + g + 8] = d.l2norm ? d.scale * rsqrtf(q1 + kDeltaEps) : d.scale;
        }
    }
    unsigned char *blk = a.blocks + ((b * d.heads_v + h) * a.nchunks + chunk) * kDcBlockBytes;
    if (tid < 64) {
        if (tid >= 32) {
            gh += sRed[0];
            gl += sRed[1];
            cut += __float_as_int(sRed[2]);
        }
        sGh[tid] = gh;
        sGl[tid] = gl;
        sN[tid] = cut;
        sBeta[tid] = be;
    }
    // whether the state is discarded in the chunk or behind it, or E leaves the range of 1 / E
    const bool direct = __syncthreads_or(tid < 64 && (cut || !(fabsf(gh + gl) <= 60.0f))) || sRed[3] == 0.0f;
    if (tid < 64) {
        // (in two factors: the sum of both parts would be rounded, 60 to 2^-19)
        const float e = cut ? 0.0f : ex2(gh) * ex2(gl);
        const float r = sR[tid];
        reinterpret_cast<float *>(blk + kDcC)[tid] = r * e;
        // the decays factor through the chunk's start where E is in range
        sF[tid] = r * (ex2(-gh) * ex2(-gl)); // (1 / w where it is not)
        sB[tid] = be * r * e;
        const bool hand = sRed[3] != 0.0f; // the next chunk's first token does not cut
        float se = sP[tid] * e;
        float we = hand && cut == sN[63] ? r * (ex2(sGh[63] - gh) * ex2(sGl[63] - gl)) : 0.0f;
        if (direct) {
            blk[kDcPow + tid] = dc_power(we);
            blk[kDcPow + 64 + tid] = dc_power(se);
            we = dc_mantissa(we);
            se = dc_mantissa(se);
            sF[tid] = 1.0f / we;
            sP[tid] = sP[tid] / se;
        }
        reinterpret_cast<float *>(blk + kDcW)[tid] = we;
        reinterpret_cast<float *>(blk + kDcS)[tid] = se;
        if (tid == 0) {
            reinterpret_cast<float *>(blk + kDcE)[0] = !hand || sN[63] ? 0.0f : ex2(sGh[63]) * ex2(sGl[63]);
            reinterpret_cast<float *>(blk + kDcE)[1] = direct ? 1.0f : 0.0f;
        }
    }
    __syncthreads();
    // ---- A, in place of K K^T, and P ---------------------------------------------------
    {
        const int i0 = 16 * warp + (lane >> 2), j0 = 2 * (lane & 3);
        // rows scale by bi (A) and pi (P'); d2(j, x) are A's factors of columns j and j + 1, and
        // those of P' in chunks with cuts or strong decays
        auto scale = [&](float2 bi, float2 pi, bool both, auto d2) {
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) {
                if (jb <= (warp | 1)) { // (above the diagonal: zeros of the slices)
                    uint32_t w[4], wl[4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int nt = 2 * jb + n, j = 8 * nt + j0;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int i = i0 + 8 * x;
                            const float b1 = x ? bi.y : bi.x, p1 = x ? pi.y : pi.x;
                            const float2 f = d2(j, x);
                            float2 av = __fmul2_rn(__fmul2_rn(f, make_float2(b1, b1)),
                                                   make_float2(kk[nt][2 * x], kk[nt][2 * x + 1]));
                            const float2 pf = make_float2(p1, p1);
                            float2 pv = make_float2(qk[nt][2 * x], qk[nt][2 * x + 1]);
                            pv = __fmul2_rn(both ? __fmul2_rn(__fmul2_rn(f, *reinterpret_cast<const float2 *>(sF + j)), pf)
                                                 : pf,
                                            pv);
                            if (jb >= warp) { // on or above the diagonal blocks
                                av.x = j < i ? av.x : 0.0f;
                                av.y = j + 1 < i ? av.y : 0.0f;
                                pv.x = j <= i ? pv.x : 0.0f;
                                pv.y = j + 1 <= i ? pv.y : 0.0f;
                            }
                            kk[nt][2 * x] = av.x;
                            kk[nt][2 * x + 1] = av.y;
                            split_bf16x2(pv.x, pv.y, w[2 * n + x], wl[2 * n + x]);
                        }
                    }
                    dp_store_block(img + 2 * kDcMat, warp, jb, lane, w);
                    dp_store_block(img + 3 * kDcMat, warp, jb, lane, wl);
                }
            }
        };
        if (!direct) {
            const float inv = ex2(-sGh[63]) * ex2(-sGl[63]); // 1 / E_63
            scale(make_float2(sB[i0], sB[i0 + 8]), make_float2(inv, inv), false,
                  [&](int j, int) { return *reinterpret_cast<const float2 *>(sF + j); });
        } else {
            const float gih[2] = {sGh[i0], sGh[i0 + 8]}, gil[2] = {sGl[i0], sGl[i0 + 8]};
            const int ni[2] = {sN[i0], sN[i0 + 8]};
            scale(make_float2(sBeta[i0] * sR[i0], sBeta[i0 + 8] * sR[i0 + 8]), make_float2(sP[i0], sP[i0 + 8]), true,
                  [&](int j, int x) {
                      return make_float2(
                          sN[j] == ni[x] ? sR[j] * ex2((gih[x] - sGh[j]) + (gil[x] - sGl[j])) : 0.0f,
                          sN[j + 1] == ni[x] ? sR[j + 1] * ex2((gih[x] - sGh[j + 1]) + (gil[x] - sGl[j + 1])) : 0.0f);
                  });
        }
    }
    // ---- T ---------------------------------------------------------------------------------
    float *sD = reinterpret_cast<float *>(dp_sm + Sm::kDiag) + warp * 16 * kDpDRow;
    float4 *sT = reinterpret_cast<float4 *>(dp_sm + Sm::kTT); // block k (k + 1) / 2 + j, then [lane][2]
    const int g = lane >> 2, t2 = 2 * (lane & 3);
    DpFrag tw; // T_ww
    {
        // the diagonal block by rows in shared memory; lane j (and j + 16) solves (I + A) x = e_j
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w == warp) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        *reinterpret_cast<float2 *>(sD + (g + 8 * x) * kDpDRow + 8 * n + t2) =
                            make_float2(kk[2 * w + n][2 * x], kk[2 * w + n][2 * x + 1]);
            }
        }
        __syncwarp();
        float x[16];
        const int j = lane & 15;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = i == j ? 1.0f : 0.0f;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
            const float4 *row = reinterpret_cast<const float4 *>(sD + i * kDpDRow);
#pragma unroll
            for (int m = 0; m < (i + 3) / 4; ++m) { // A is 0 on and above the diagonal
                const float4 v = row[m];
                s0 = __ffma2_rn(make_float2(v.x, v.y), make_float2(x[4 * m], x[4 * m + 1]), s0);
                s1 = __ffma2_rn(make_float2(v.z, v.w), make_float2(x[4 * m + 2], x[4 * m + 3]), s1);
            }
            x[i] -= (s0.x + s0.y) + (s1.x + s1.y);
        }
        __syncwarp();
        // column j as row j: the transpose
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4 *>(sD + j * kDpDRow + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        }
        __syncwarp();
        DpFrag tt;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int xx = 0; xx < 2; ++xx) {
                const float2 v = *reinterpret_cast<const float2 *>(sD + (g + 8 * xx) * kDpDRow + 8 * n + t2);
                tt.f[4 * n + 2 * xx] = v.x;
                tt.f[4 * n + 2 * xx + 1] = v.y;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    tw.f[4 * n + 2 * xx + e] = sD[(8 * n + t2 + e) * kDpDRow + g + 8 * xx];
            }
        if (warp < 3) {
            float4 *dst = sT + (warp * (warp + 1) / 2 + warp) * 64 + lane;
            dst[0] = make_float4(tt.f[0], tt.f[1], tt.f[2], tt.f[3]);
            dst[32] = make_float4(tt.f[4], tt.f[5], tt.f[6], tt.f[7]);
        }
    }
    // T_wj diag(beta), split, into the image
    auto put = [&](int jb, const DpFrag &t) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float2 bj = *reinterpret_cast<const float2 *>(sBeta + 16 * jb + 8 * n + t2);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float2 v = __fmul2_rn(bj, make_float2(t.f[4 * n + 2 * x], t.f[4 * n + 2 * x + 1]));
                split_bf16x2(v.x, v.y, hi[2 * n + x], lo[2 * n + x]);
            }
        }
        dp_store_block(img, warp, jb, lane, hi);
        dp_store_block(img + kDcMat, warp, jb, lane, lo);
    };
    put(warp, tw);
    const DpOp to = dp_split(tw);
    if (!(warp & 1)) { // the block above the diagonal one in the slices: zeros
        const uint32_t zero[4] = {0u, 0u, 0u, 0u};
        dp_store_block(img, warp, warp + 1, lane, zero);
        dp_store_block(img + kDcMat, warp, warp + 1, lane, zero);
    }
#pragma unroll
    for (int step = 1; step < 4; ++step) {
        __syncthreads(); // the T_kj^T with k - j < step are there
        if (warp >= step) {
            const int j = warp - step;
            DpFrag wt = {};
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (k >= j && k < warp) {
                    const float4 *src = sT + (k * (k + 1) / 2 + j) * 64 + lane;
                    const float4 u = src[0], v = src[32];
                    const DpFrag tt = {{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w}};
                    const DpFrag ak = {{kk[2 * k][0], kk[2 * k][1], kk[2 * k][2], kk[2 * k][3], kk[2 * k + 1][0],
                                        kk[2 * k + 1][1], kk[2 * k + 1][2], kk[2 * k + 1][3]}};
                    dp_mul(wt, dp_split(tt), dp_split(ak));
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                wt.f[i] = -wt.f[i];
            const DpOp wo = dp_split(wt);
            DpFrag x = {};
            dp_mul(x, to, wo);
            put(j, x);
            if (warp < 3) {
                DpFrag xt = {};
                dp_mul(xt, wo, to);
                float4 *dst = sT + (warp * (warp + 1) / 2 + j) * 64 + lane;
                dst[0] = make_float4(xt.f[0], xt.f[1], xt.f[2], xt.f[3]);
                dst[32] = make_float4(xt.f[4], xt.f[5], xt.f[6], xt.f[7]);
            }
        }
    }
    // ---- the matrices of the block ------------------------------------------------------
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(blk + kDcThi), "r"(img),
                     "r"(2 * kDcMat)
                     : "memory");
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(blk + kDcP),
                     "r"(img + 2 * kDcMat), "r"(2 * kDcMat)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
    }
}

// ---- the walk ------------------------------------------------------------------------

// What bounds it is the chain of hand-overs from one product to the next (KH^T, R, U, dH, H),
// chunk after chunk.  256 walks of 32 chunks (8 x 2048 tokens x 32 heads of 128 x 128) take
// 169-178 us, two an SM, and 189 us where an eighth of the heads decays strongly: tensor cores
// busy 35% of the time, instructions issued in 41% of the cycles, 497 MB read and 124 MB
// written.  Alone on its SM a walk of 32 chunks takes 100 us, 3.1 us a chunk.  (Two walks an SM
// without any element-wise work took 89 us of the 170 us of a walk with fewer products.)
//
// G: groups of four compute warps, each with a G-th of the columns: 2 (two CTAs per SM) or
// 4 (one CTA per SM).  A CTA alone on its SM has room for Y^T beside the rest, in two places
// that alternate: H^T Q^T follows KH^T at once, (w o U)^T P'^T follows dH^T, and the outputs
// leave after the state is handed on, while the next chunk's first product runs.  With two CTAs
// Y^T takes R^T's place, between U^T and dH^T.
template <int G> struct DwShape {
    static constexpr int kWarps = 4 * G;              // compute warps
    static constexpr int kThreads = 32 * kWarps + 32; // + the issuer warp
    static constexpr int kCtas = G == 2 ? 2 : 1;      // per SM
    static constexpr int kTok = kDcChunk / G, kKeys = 128 / G; // columns of a warp: tokens, keys
    static constexpr bool kLate = G == 4;
    static constexpr uint32_t kCols = kLate ? 512 : 256; // tensor memory
    static constexpr uint32_t kY = kLate ? 256 : 128;    // Y^T
    static constexpr uint32_t kYStep = kLate ? 64 : 0;   // from Y^T of even chunks to that of odd ones
};
// tensor-memory columns.  H: 16 columns per 16 keys, the high parts of H^T in the first
// 8 (packed pairs), the remainders in the last 8; dH^T is accumulated over them.  D1: KH^T,
// then R^T over it in the same form (16 columns per 16 tokens).  D2: U^T, then
// (w o U)^T over it.
constexpr uint32_t kDwH = 0, kDwD1 = 128, kDwD2 = 192;

template <int G> struct DwSmem { // from a 1024-byte aligned base
    static constexpr int kK = 0;                // k chunk: 2 stages of two [64 tokens x 64 keys] tiles
    static constexpr int kQ = kK + 2 * 16384;   // q chunk: two tiles
    static constexpr int kV = kQ + 16384;       // v chunk: two [64 tokens x 64 values] tiles
    static constexpr int kB = kV + 16384;       // workspace blocks up to P': 2 stages
    static constexpr int kP = kB + 2 * kDcHead; // P' hi, P' lo
    // outputs: a tile of [kTok tokens x 32 values] per compute warp, with two CTAs an SM in the
    // place of the q chunk, which has been read by then
    static constexpr int kY = DwShape<G>::kLate ? kP + 2 * kDcMat : kQ;
    static constexpr int kBar = kP + 2 * kDcMat + (DwShape<G>::kLate ? 16384 : 0);
    static constexpr int kTmem = kBar + 144;
    static constexpr int kAlive = kTmem + 4;  // the walk for M: chunks after which it was not 0
    static constexpr int kDone = kAlive + 4;  // and whether it has become 0
    static constexpr int kBad = kDone + 4;    // the state or an output is not finite (walks with outputs)
    static constexpr int kBytes = kBar + 256;
};
// two CTAs on an SM: 228 KB, 1 KB of it reserved for each
static_assert(DwSmem<2>::kBytes <= 113 * 1024 && DwSmem<4>::kBytes <= 227 * 1024, "shared memory of the walk");

struct DeltaWalkArgs {
    DeltaArgs d; // as called: for the columns that are walked token by token
    int64_t batch;
    int seq, heads_v, ratio, dk, dv;
    int nchunks, col_tiles, nks;  // nks: 16-key slices of the state
    int segments, seg_chunks;     // 1 segment: one pass over all chunks
    int pass;                     // 0, or 1 and 2 (see above)
    float *seg_n;                 // [batch, heads_v, segments - 1, dk, dv]: N, then the state after the segment
    float *seg_h0;                // [batch, heads_v, dk, dv]: pass 1's copy of h0, which pass 2 reads when the
                                  // final state takes h0's place; null otherwise
    float *seg_m;                 // [batch, heads_v, segments - 2, dk, dk]: M of segments 1 ..
    int *seg_zero;                // [batch, heads_v, segments - 2]: 1 where M is 0 (and not written)
    int hold;                     // failure-path test aid: withhold the first arrivals on arr_r
    const unsigned char *blocks;
    const float *h0;              // nullable
    const float *g;               // nullable; g and reset for the first token
    const uint8_t *reset;         // nullable
    __nv_bfloat16 *y;
    float *final_state;           // nullable
};

struct DeltaWalkMaps {
    CUtensorMap q, k, v; // 4-D (d, head, token, batch), boxes (64, 1, 64, 1)
};

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
                 : "memory");
}
// Matrix descriptor of K-major rows of 32 bytes in the 32-byte swizzle (layout type 6),
// 8-row groups 256 bytes apart.
__device__ __forceinline__ uint64_t sw32_desc(uint32_t saddr)
{
    return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(256 >> 4) << 32) | (uint64_t(1) << 46) |
           (uint64_t(6) << 61);
}

// A pair of values split into high parts and remainders, as split_bf16x2 does, with one
// packed subtraction.
__device__ __forceinline__ void dw_split2(float2 x, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x.x, x.y);
    const float2 r = __ffma2_rn(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)),
                                make_float2(-1.0f, -1.0f), x);
    lo = pack_bf16x2(r.x, r.y);
}

// (exact for a power of two)
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float2 dw_pair(const uint32_t (&r)[8], int e)
{
    return make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
}

// One thread of a converged warp, chosen by the hardware: the compiler then knows that
// one thread issues, and keeps the operands of tcgen05.mma in uniform registers.  (An MMA
// of N = 64 takes 33 cycles so, and 48 when the thread is picked by its index; N = 32, 18
// and 48.)
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// The element-wise steps hold tiles of 16 lanes as the warp-wide fragments that
// tcgen05.ld.16x256b, tcgen05.st.16x128b, ldmatrix and stmatrix share: thread t has rows
// t / 4 and t / 4 + 8 (x = 0, 1), and of every 8 columns the pair 2 (t % 4), + 1.
// 16 fp32 columns: r[4 k + 2 x + e] is column 8 k + 2 (t % 4) + e.  (Not 32: eight more
// registers beside H would spill.)
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
    tmem_ld_wait();
    // (the registers are only valid once the wait has returned)
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
}
// 16 columns of packed pairs, those of 8 k in columns 4 k .. : r[2 k + x]
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t saddr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t saddr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// The columns n0 .. n0 + 127 of segment `seg` once more, token by token in fp32, where the
// walk's state or an output has become infinite or NaN.  In products over a chunk 0 times such
// a value reaches tokens that do not depend on it (those before it, and those behind a reset);
// it then always stays in the state, which the walk looks at once, at its end.  Outputs are
// looked at as they leave, since they can pass the range of fp32 on the way to finite values:
// (w o U)^T P'^T is up to 2^60 times what it stands for.  Here a token only meets what it
// depends on.  From the state after the segment before when that is finite, or from the first
// token.  Two syncs a token, two threads a column, the state in shared memory: 2.6 us a token
// (5.2 ms for 2048 tokens), for inputs that hold or lead to such values only.
__device__ __noinline__ void delta_rewalk(const DeltaWalkArgs &a, unsigned char *sm, int64_t bh, int seg, int n0)
{
    const DeltaArgs &d = a.d;
    float *st = reinterpret_cast<float *>(sm);              // [dk][128]
    float *kq = st + 128 * 128;                             // two of k[128], q[128], (decay, beta, q . k)
    float *part = kq + 2 * 264;                             // [2 halves][k . S, q . S][128]
    const int tid = threadIdx.x, lane = tid & 31, col = tid & 127, half = tid >> 7;
    const bool mine = tid < 256, in = n0 + col < a.dv;
    const int64_t b = bh / a.heads_v;
    const int h = int(bh % a.heads_v), hk = h / a.ratio;
    const int k0 = half ? d.dk / 2 : 0, k1 = half ? d.dk : d.dk / 2; // this thread's keys
    const int64_t ofs = bh * a.dk * a.dv + n0 + col;
    auto load = [&](const float *from) {
        bool bad = false;
        for (int i = k0; mine && i < k1; ++i) {
            const float x = from && in ? from[int64_t(i) * a.dv] : 0.0f;
            bad = bad || !(fabsf(x) < INFINITY);
            st[i * 128 + col] = x;
        }
        return __syncthreads_or(bad);
    };
    int64_t t = int64_t(seg) * a.seg_chunks * kDcChunk;
    const int64_t first = t, last = t + int64_t(a.seg_chunks) * kDcChunk, end = last < a.seq ? last : a.seq;
    const float *h0 = a.pass == 2 && a.seg_h0 ? a.seg_h0 : a.h0;
    if (seg == 0 || load(a.seg_n + (bh * (a.segments - 1) + seg - 1) * a.dk * a.dv + n0 + col)) {
        t = 0;
        load(h0 ? h0 + ofs : nullptr);
    }
    // the first warp reads the next token's rows and gates, and everyone its value, ahead
    __nv_bfloat16 q[4], k[4], vn = __float2bfloat16_rn(0.0f);
    float gn = 1.0f, bn = 1.0f;
    const int64_t ch = int64_t(h) * a.dv + n0 + col;
    auto fetch = [&](int64_t pos) {
        const int64_t tok = b * a.seq + pos;
        if (tid < 32) {
            const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(d.q) + tok * d.q_stride + int64_t(hk) * d.dk;
            const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(d.k) + tok * d.k_stride + int64_t(hk) * d.dk;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = lane + 32 * j;
                q[j] = i < d.dk ? qp[i] : __float2bfloat16_rn(0.0f);
                k[j] = i < d.dk ? kp[i] : __float2bfloat16_rn(0.0f);
            }
            const int64_t gi = tok * a.heads_v + h;
            gn = d.reset && d.reset[tok] ? -INFINITY : d.g ? d.g[gi] : 0.0f;
            bn = d.beta ? d.beta[gi] : 1.0f;
        }
        if (mine && in)
            vn = static_cast<const __nv_bfloat16 *>(d.v)[tok * d.v_stride + ch];
    };
    fetch(t);
    for (; t < end; ++t) {
        float *buf = kq + (t & 1) * 264;
        if (tid < 32) {
            float qf[4], kf[4], qq = 0.0f, kk = 0.0f, qk = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                qf[j] = __bfloat162float(q[j]);
                kf[j] = __bfloat162float(k[j]);
                qq = fmaf(qf[j], qf[j], qq);
                kk = fmaf(kf[j], kf[j], kk);
                qk = fmaf(qf[j], kf[j], qk);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                qq += __shfl_xor_sync(0xffffffffu, qq, o);
                kk += __shfl_xor_sync(0xffffffffu, kk, o);
                qk += __shfl_xor_sync(0xffffffffu, qk, o);
            }
            const float rq = d.l2norm ? d.scale * rsqrtf(qq + kDeltaEps) : d.scale;
            const float rk = d.l2norm ? rsqrtf(kk + kDeltaEps) : 1.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                buf[lane + 32 * j] = rk * kf[j];
                buf[128 + lane + 32 * j] = rq * qf[j];
            }
            if (lane == 0) {
                buf[256] = expf(gn);
                buf[257] = bn;
                buf[258] = qk * rq * rk;
            }
        }
        const float v = __bfloat162float(vn);
        __syncthreads();
        if (t + 1 < end)
            fetch(t + 1);
        const float decay = buf[256];
        if (mine) {
            float ks = 0.0f, qs = 0.0f;
            if (decay != 0.0f) { // a decay of 0 discards the state, whatever it holds
#pragma unroll 8
                for (int i = k0; i < k1; ++i) {
                    const float x = st[i * 128 + col];
                    ks = fmaf(buf[i], x, ks);
                    qs = fmaf(buf[128 + i], x, qs);
                }
            }
            part[half * 256 + col] = ks;
            part[half * 256 + 128 + col] = qs;
        }
        __syncthreads();
        if (mine) {
            const float ks = decay * (part[col] + part[256 + col]), qs = decay * (part[128 + col] + part[384 + col]);
            const float u = buf[257] * (v - ks);
            for (int i = k0; i < k1; i += 4) { // (dk is a multiple of 8; reads before writes)
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = fmaf(buf[i + e], u, decay == 0.0f ? 0.0f : decay * st[(i + e) * 128 + col]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    st[(i + e) * 128 + col] = x[e];
            }
            if (half == 0 && in && t >= first)
                a.y[(b * a.seq + t) * a.heads_v * a.dv + ch] = __float2bfloat16_rn(fmaf(buf[258], u, qs));
        }
    }
    if (a.final_state && seg == a.segments - 1)
        for (int i = k0; mine && in && i < k1; ++i)
            a.final_state[ofs + int64_t(i) * a.dv] = st[i * 128 + col];
}

template <int G>
__global__ void __launch_bounds__(DwShape<G>::kThreads, DwShape<G>::kCtas)
ss_delta_walk_kernel(const __grid_constant__ DeltaWalkArgs a, const __grid_constant__ DeltaWalkMaps maps, uint32_t *status)
{
    using Sh = DwShape<G>;
    using Sm = DwSmem<G>;
    constexpr int kWarps = Sh::kWarps, kTok = Sh::kTok, kKeys = Sh::kKeys;
    constexpr bool kLate = Sh::kLate;
    extern __shared__ __align__(1024) unsigned char dw_sm[];
    unsigned char *sm = dw_sm;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Sm::kBar);
    // loads (k, workspace block: two stages each), products, and the compute warps' arrivals
    uint64_t *bar_k = bars, *bar_b = bars + 2, *bar_q = bars + 4, *bar_v = bars + 5, *bar_p = bars + 6,
             *bar_kh = bars + 7, *bar_u = bars + 8, *bar_qh = bars + 9, *bar_y = bars + 10, *bar_dh = bars + 11 /* [2] */;
    uint64_t *arr_h = bars + 13, *arr_q = bars + 14, *arr_r = bars + 15, *arr_u = bars + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + Sm::kTmem);
    volatile int *s_alive = reinterpret_cast<int *>(sm + Sm::kAlive);
    volatile int *s_done = reinterpret_cast<int *>(sm + Sm::kDone);
    volatile int *s_bad = reinterpret_cast<int *>(sm + Sm::kBad);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const bool issuer = warp == kWarps;
    // (head, segment, column tile); tile col_tiles of pass 1 is the walk for M
    int tile, seg = 0;
    int64_t bh;
    if (a.pass == 1) {
        const unsigned per = unsigned(a.col_tiles + (a.segments - 2) * (a.col_tiles + 1));
        bh = blockIdx.x / per;
        tile = int(blockIdx.x % per);
        if (tile >= a.col_tiles) {
            seg = 1 + (tile - a.col_tiles) / (a.col_tiles + 1);
            tile = (tile - a.col_tiles) % (a.col_tiles + 1);
        }
    } else {
        const unsigned per = unsigned(a.segments * a.col_tiles);
        bh = blockIdx.x / per;
        seg = int(blockIdx.x % per) / a.col_tiles;
        tile = int(blockIdx.x % per) % a.col_tiles;
    }
    const bool outs = a.pass != 1, for_m = tile == a.col_tiles;
    const int64_t b = bh / a.heads_v;
    const int h = int(bh % a.heads_v), hk = h / a.ratio;
    const int n0 = for_m ? 0 : 128 * tile;
    const int cols = for_m ? a.dk : a.dv; // columns of the state walked
    const int cb = seg * a.seg_chunks;    // the segment's chunks: cb + c, c < nc
    const int nc = a.nchunks - cb < a.seg_chunks ? a.nchunks - cb : a.seg_chunks;
    const uint32_t s_base = smem_u32(sm);

    if (tid == 0) {
        for (int i = 0; i < 13; ++i)
            mbar_init(bars + i, 1);
        for (int i = 13; i < 17; ++i)
            mbar_init(bars + i, kWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *s_alive = *s_done = *s_bad = 0;
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, Sh::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(tmem_slot), 0);
    // (the swizzled tiles need a 1024-byte aligned base; shared memory starts at one)
    bool ok = (s_base & 1023u) == 0;
    if (!ok && tid == 0)
        atomicOr(status, 1u << kStatusTimeout);

    int failed = !ok; // a wait ran out
    if (ok && issuer) {
        // ======================= the issuer warp (one thread works) =======================
        if (elect_one()) {
            const int32_t b32 = int32_t(b);
            const unsigned char *blocks = a.blocks + (bh * a.nchunks + cb) * kDcBlockBytes;
            const int t_first = cb * kDcChunk;
            // barriers with a phase begun by a load or a product, and its parity
            uint32_t begun = 0, latest = ~0u;
            auto begin = [&](const uint64_t *bar) {
                begun |= 1u << int(bar - bars);
                latest ^= 1u << int(bar - bars);
            };
            auto commit = [&](uint64_t *bar) {
                umma_commit(bar);
                begin(bar);
            };
            auto load_kb = [&](int c) {
                const int st = c & 1, t = t_first + c * kDcChunk;
                begin(bar_k + st);
                begin(bar_b + st);
                mbar_arrive_expect_tx(bar_k + st, 16384);
                tma_load_4d(sm + Sm::kK + st * 16384, &maps.k, 0, hk, t, b32, bar_k + st);
                tma_load_4d(sm + Sm::kK + st * 16384 + 8192, &maps.k, 64, hk, t, b32, bar_k + st);
                mbar_arrive_expect_tx(bar_b + st, kDcHead);
                bulk_load(sm + Sm::kB + st * kDcHead, blocks + int64_t(c) * kDcBlockBytes, kDcHead, bar_b + st);
            };
            auto load_p = [&](int c) {
                begin(bar_p);
                mbar_arrive_expect_tx(bar_p, 2 * kDcMat);
                bulk_load(sm + Sm::kP, blocks + int64_t(c) * kDcBlockBytes + kDcP, 2 * kDcMat, bar_p);
            };
            auto load_q = [&](int c) {
                begin(bar_q);
                mbar_arrive_expect_tx(bar_q, 16384);
                tma_load_4d(sm + Sm::kQ, &maps.q, 0, hk, t_first + c * kDcChunk, b32, bar_q);
                tma_load_4d(sm + Sm::kQ + 8192, &maps.q, 64, hk, t_first + c * kDcChunk, b32, bar_q);
            };
            auto load_v = [&](int c) {
                begin(bar_v);
                mbar_arrive_expect_tx(bar_v, 16384);
                tma_load_4d(sm + Sm::kV, &maps.v, n0, h, t_first + c * kDcChunk, b32, bar_v);
                tma_load_4d(sm + Sm::kV + 8192, &maps.v, n0 + 64, h, t_first + c * kDcChunk, b32, bar_v);
            };
            constexpr uint32_t kIdTok = idesc_bf16(128, kDcChunk, 0, 0), kIdHalf = idesc_bf16(128, 32, 0, 0);
            // dH in halves of 64 keys
            const int nk0 = a.nks < 4 ? a.nks : 4;
            const uint32_t id_dh0 = idesc_bf16(128, 16 * nk0, 0, 1), id_dh1 = idesc_bf16(128, 16 * (a.nks - nk0), 0, 1);
            load_kb(0);
            if (!for_m)
                load_v(0);
            if (outs) {
                load_q(0);
                load_p(0);
            }
            if (nc > 1)
                load_kb(1);
            // H^T Q^T into Y^T
            auto mul_qh = [&](uint32_t dy) {
                for (int ks = 0; ks < a.nks; ++ks) {
                    const uint64_t qd = sw128_desc(s_base + Sm::kQ + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024);
                    umma_bf16_ts(dy, tmem + kDwH + 16 * ks, qd, kIdTok, ks > 0);
                    umma_bf16_ts(dy, tmem + kDwH + 16 * ks + 8, qd, kIdTok, 1);
                }
                commit(bar_qh);
            };
            // + (w o U)^T P'^T, in halves of another shape: after H^T Q^T has completed
            auto mul_up = [&](uint32_t dy) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int ks = 0; ks < 2 + 2 * hf; ++ks) {
                        const uint32_t uh = tmem + kDwD2 + 16 * ks;
                        const uint32_t at = s_base + Sm::kP + dc_slice(ks) + (ks < 2 ? 1024 * hf : 0);
                        const uint64_t ph = sw32_desc(at), pl = sw32_desc(at + kDcMat);
                        umma_bf16_ts(dy + 32 * hf, uh, ph, kIdHalf, 1);
                        umma_bf16_ts(dy + 32 * hf, uh + 8, ph, kIdHalf, 1);
                        umma_bf16_ts(dy + 32 * hf, uh, pl, kIdHalf, 1);
                    }
                commit(bar_y);
            };
            for (int c = 0; c < nc; ++c) {
                const int st = c & 1;
                const uint32_t ph = uint32_t(c & 1), ph2 = uint32_t((c >> 1) & 1);
                const uint32_t d1 = tmem + kDwD1, dy = tmem + Sh::kY + (c & 1) * Sh::kYStep;
                const uint32_t kb = s_base + Sm::kK + st * 16384, bb = s_base + Sm::kB + st * kDcHead;
                // KH^T once the tile has landed and H(c) is written
                if (!mbar_wait(bar_k + st, ph2, status) || !mbar_wait(arr_h, ph, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (for_m && c > 0 && *s_alive != c) { // 0 from here on
                    *s_done = 1;
                    begin(bar_kh);
                    mbar_arrive(bar_kh);
                    break;
                }
                for (int ks = 0; ks < a.nks; ++ks) {
                    const uint64_t kd = sw128_desc(kb + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024);
                    umma_bf16_ts(d1, tmem + kDwH + 16 * ks, kd, kIdTok, ks > 0);
                    umma_bf16_ts(d1, tmem + kDwH + 16 * ks + 8, kd, kIdTok, 1);
                }
                commit(bar_kh);
                // the product that reads P has completed
                if (c > 0 && outs) {
                    if (!mbar_wait(bar_y, ph ^ 1, status)) {
                        ok = false;
                        break;
                    }
                    load_p(c);
                    if (!kLate) // the outputs of c - 1 have left its place (before H(c) was written)
                        load_q(c);
                }
                if (outs && kLate) {
                    if (!mbar_wait(bar_q, ph, status) || !mbar_wait(arr_q, ph, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mul_qh(dy);
                }
                // U^T once R is written: the blocks of T on and below the diagonal
                if (!mbar_wait(bar_b + st, ph2, status) || !mbar_wait(arr_r, ph, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                    for (int ks = 0; ks < 2 + 2 * hf; ++ks) {
                        const uint32_t dst = tmem + kDwD2 + 32 * hf, rhi = d1 + 16 * ks, rlo = rhi + 8;
                        const uint32_t to = bb + dc_slice(ks) + (ks < 2 ? 1024 * hf : 0);
                        const uint64_t thi = sw32_desc(to + kDcThi), tlo = sw32_desc(to + kDcTlo);
                        umma_bf16_ts(dst, rhi, thi, kIdHalf, ks > 0);
                        umma_bf16_ts(dst, rlo, thi, kIdHalf, 1);
                        umma_bf16_ts(dst, rhi, tlo, kIdHalf, 1);
                    }
                }
                commit(bar_u);
                // the other stage: dH(c - 1) has completed (before H(c) was written) and the
                // outputs of c - 1 have left (before R(c) was written)
                if (c > 0 && c + 1 < nc)
                    load_kb(c + 1);
                if (c + 1 < nc && !for_m) // R(c), the only reader of v, is written
                    load_v(c + 1);
                if (outs && kLate) {
                    if (!mbar_wait(bar_qh, ph, status)) { // (long done)
                        ok = false;
                        break;
                    }
                    if (c + 1 < nc)
                        load_q(c + 1);
                }
                if (outs && !kLate) { // Y^T over R, once R has been read
                    if (!mbar_wait(bar_q, ph, status) || !mbar_wait(arr_q, ph, status) ||
                        !mbar_wait(bar_u, ph, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mul_qh(dy);
                }
                // w o U is written: dH^T over H, which has been read
                if (!mbar_wait(arr_u, ph, status) || (outs && !mbar_wait(bar_p, ph, status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (outs && !kLate) {
                    if (!mbar_wait(bar_qh, ph, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mul_up(dy);
                }
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t kd = sw128_desc(kb + ks * 2048, 8192, 1024); // keys x 16 tokens (MN-major)
                    umma_bf16_ts(tmem + kDwH, tmem + kDwD2 + 16 * ks, kd, id_dh0, ks > 0);
                    umma_bf16_ts(tmem + kDwH, tmem + kDwD2 + 16 * ks + 8, kd, id_dh0, 1);
                }
                commit(bar_dh);
                if (a.nks > 4) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t kd = sw128_desc(kb + 8192 + ks * 2048, 8192, 1024);
                        umma_bf16_ts(tmem + kDwH + 64, tmem + kDwD2 + 16 * ks, kd, id_dh1, ks > 0);
                        umma_bf16_ts(tmem + kDwH + 64, tmem + kDwD2 + 16 * ks + 8, kd, id_dh1, 1);
                    }
                }
                commit(bar_dh + 1);
                if (outs && kLate)
                    mul_up(dy);
            }
            // let every load and product in flight finish before the tensor memory is freed:
            // the latest phase of each barrier
            for (int i = 0; i < 13; ++i)
                if ((begun >> i) & 1u)
                    mbar_wait(bars + i, (latest >> i) & 1u, nullptr);
        }
        __syncwarp();
        failed = __syncthreads_or(!ok);
    } else if (ok) {
        // ======================= the compute warps =======================================
        // warp w: two tiles m of 16 tensor-memory lanes from row0, group cg of the columns (keys
        // kKeys cg .. of H, tokens kTok cg .. of the chunk)
        const int row0 = 32 * (warp & 3), cg = warp >> 2;
        const int tr = lane >> 2, tc = 2 * (lane & 3); // this thread's row and column pair of a fragment
        const int col = n0 + row0 + tr;             // its first value column; the others 8 apart
        const uint32_t lanes = tmem + (uint32_t(row0) << 16);
        // H[m][k][x]: value column col + 16 m + 8 x, keys kKeys cg + 8 k + tc, + 1
        float2 H[2][kKeys / 8][2];
        bool zero = false; // M has become 0
        // the state the segment starts from: h0, the state after the segment before it, the
        // identity, or zero
        const float *from = nullptr;
        if (a.pass == 2 && seg > 0)
            from = a.seg_n + (bh * (a.segments - 1) + seg - 1) * a.dk * a.dv;
        else if (seg == 0 && a.h0 && !dc_cut(a.reset, a.g, b * a.seq, a.heads_v, h))
            from = (a.pass == 2 && a.seg_h0 ? a.seg_h0 : a.h0) + bh * a.dk * a.dv;
        const int64_t sofs = int64_t(kKeys * cg + tc) * cols + col;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < kKeys / 8; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int key = kKeys * cg + 8 * k + tc, vc = col + 16 * m + 8 * x;
                    const bool in = from && key < a.dk && vc < cols; // (dk is even)
                    const int64_t o = sofs + int64_t(8 * k) * cols + 16 * m + 8 * x;
                    H[m][k][x] = make_float2(in ? from[o] : 0.0f, in ? from[o + cols] : 0.0f);
                    if (for_m && key < a.dk) // the identity (padded keys are never updated: they stay 0)
                        H[m][k][x] = make_float2(key == vc ? 1.0f : 0.0f, key + 1 == vc ? 1.0f : 0.0f);
                    if (in && a.pass == 1 && seg == 0 && a.seg_h0) {
                        a.seg_h0[bh * a.dk * a.dv + o] = H[m][k][x].x;
                        a.seg_h0[bh * a.dk * a.dv + o + cols] = H[m][k][x].y;
                    }
                }
        // 16 keys (2 k-blocks from kb) of tile m as operand columns
        auto store_h = [&](int m, int kb) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    dw_split2(H[m][kb + i][x], w[2 * i + x], w[4 + 2 * i + x]);
            tmem_st_frag(lanes + (uint32_t(16 * m) << 16) + kDwH + kKeys * cg + 8 * kb, w);
        };
        auto arrive = [&](uint64_t *bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar);
        };
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            const bool good = __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
            tc_fence_after();
            return good;
        };
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int kb = 0; kb < kKeys / 8; kb += 2)
                store_h(m, kb);
        tmem_st_wait();
        arrive(arr_h);
        const uint32_t v_base = s_base + Sm::kV + (row0 >> 6) * 8192; // the tile of this warp's values
        unsigned char *ytile = sm + Sm::kY + warp * (64 * kTok);
        const uint32_t y_base = smem_u32(ytile);
        // this lane's 16 bytes of the tile's first eight rows; eight rows further on, ystep more
        const int64_t ystep = int64_t(8) * a.heads_v * a.dv;
        __nv_bfloat16 *yp = a.y + ((b * a.seq + cb * kDcChunk + kTok * cg + (lane >> 2)) * a.heads_v + h) * a.dv + n0 + row0 +
                            8 * (lane & 3);
        for (int c = 0; c < nc; ++c) {
            const int st = c & 1;
            const uint32_t ph = uint32_t(c & 1), ph2 = uint32_t((c >> 1) & 1);
            const unsigned char *blk = sm + Sm::kB + st * kDcHead;
            const float *sc = reinterpret_cast<const float *>(blk + kDcC) + kTok * cg + tc;
            const float *sw = reinterpret_cast<const float *>(blk + kDcW) + kTok * cg + tc;
            const float *ss_ = reinterpret_cast<const float *>(blk + kDcS);
            // the shared-memory addresses of a step are computed when it runs: kept over the
            // loop they would cost the registers that H needs
            int ln = lane;
            asm volatile("" : "+r"(ln));
            if (!wait(bar_b + st, ph2)) {
                ok = false;
                break;
            }
            const float2 em = *reinterpret_cast<const float2 *>(blk + kDcE); // E_63, mode
            // ---- rows of K (which 0) or Q (1) scaled by powers of two in place, in chunks with cuts
            // or strong decays
            auto scale = [&](int from, int to) {
#pragma unroll 1
                for (int which = from; which < to; ++which) {
                    if (!wait(which ? bar_q : bar_k + st, which ? ph : ph2))
                        return false;
                    unsigned char *tiles = sm + (which ? Sm::kQ : Sm::kK + st * 16384);
                    const unsigned char *pow = blk + kDcPow + 64 * which;
#pragma unroll 4
                    for (int i = 0; i < 1024 / (32 * kWarps); ++i) {
                        const int e = 32 * (kWarps * i + warp) + ln; // 16-byte chunk: tile, token, position
                        const uint32_t f = uint32_t(pow[(e >> 3) & 63]) * 0x00800080u; // the power as two bf16
                        uint4 *p = reinterpret_cast<uint4 *>(tiles + 16 * e);
                        const uint4 v = *p;
                        *p = make_uint4(mul_bf16x2(v.x, f), mul_bf16x2(v.y, f), mul_bf16x2(v.z, f), mul_bf16x2(v.w, f));
                    }
                }
                fence_proxy_async_smem();
                return true;
            };
            if (kLate && outs && em.y != 0.0f && !scale(1, 2)) {
                ok = false;
                break;
            }
            if (kLate)
                arrive(arr_q);
            // ---- R^T = V^T - KH^T diag(c) -------------------------------------------------
            if ((!for_m && !wait(bar_v, ph)) || !wait(bar_kh, ph)) {
                ok = false;
                break;
            }
            if (for_m && *s_done) {
                zero = true;
                break;
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t at = lanes + (uint32_t(16 * m) << 16) + kDwD1 + kTok * cg;
#pragma unroll
                for (int j = 0; j < kTok / 16; ++j) { // 16 tokens
                    uint32_t r[8], v[4] = {}, w[8];
                    // 8 values x 8 tokens a matrix: x = matrix % 2, token block 2 j + matrix / 2
                    if (!for_m)
                        ldmatrix_x4_trans(v, v_base + sw128_off(kTok * cg + 16 * j + 8 * (ln >> 4) + (ln & 7),
                                                                ((row0 & 63) >> 3) + 2 * m + ((ln >> 3) & 1)));
                    tmem_ld_frag(at + 16 * j, r);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 cv = *reinterpret_cast<const float2 *>(sc + 16 * j + 8 * i);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t vv = v[2 * i + x];
                            dw_split2(__ffma2_rn(make_float2(-cv.x, -cv.y), dw_pair(r, 2 * i + x),
                                                 make_float2(__uint_as_float(vv << 16), __uint_as_float(vv & 0xffff0000u))),
                                      w[2 * i + x], w[4 + 2 * i + x]);
                        }
                    }
                    tmem_st_frag(at + 16 * j, w);
                }
            }
            tmem_st_wait();
            if (!(a.hold && c == 0))
                arrive(arr_r);
            // (K H^T is done; all of this while U^T runs)
            if (em.y != 0.0f && !scale(0, !kLate && outs ? 2 : 1)) {
                ok = false;
                break;
            }
            if (!kLate)
                arrive(arr_q);
            // ---- w o U over U^T --------------------------------------------------------------
            if (!wait(bar_u, ph)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t at = lanes + (uint32_t(16 * m) << 16) + kDwD2 + kTok * cg;
#pragma unroll
                for (int j = 0; j < kTok / 16; ++j) {
                    uint32_t r[8], w[8];
                    tmem_ld_frag(at + 16 * j, r);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 wv = *reinterpret_cast<const float2 *>(sw + 16 * j + 8 * i);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            dw_split2(__fmul2_rn(wv, dw_pair(r, 2 * i + x)), w[2 * i + x], w[4 + 2 * i + x]);
                    }
                    tmem_st_frag(at + 16 * j, w);
                }
            }
            tmem_st_wait();
            arrive(arr_u);
            // ---- the outputs: while dH^T runs, or once the state is handed on -----------------
            auto emit = [&]() {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
#pragma unroll
                    for (int j = 0; j < kTok / 16; ++j) {
                        uint32_t r[8], o[4];
                        float2 zero2 = make_float2(0.0f, 0.0f);
                        tmem_ld_frag(lanes + (uint32_t(16 * m) << 16) + Sh::kY + (c & 1) * Sh::kYStep + kTok * cg + 16 * j,
                                     r);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 sv = *reinterpret_cast<const float2 *>(ss_ + kTok * cg + 16 * j + 8 * i + tc);
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float2 y = __fmul2_rn(sv, dw_pair(r, 2 * i + x));
                                zero2 = __ffma2_rn(make_float2(0.0f, 0.0f), y, zero2);
                                o[2 * i + x] = pack_bf16x2(y.x, y.y);
                            }
                        }
                        if (zero2.x + zero2.y != 0.0f) // (0 y is 0 for finite y alone)
                            *s_bad = 1;
                        // rows of 64 bytes in the 64-byte swizzle: token 8 (2 j + matrix / 2) + lane % 8,
                        // values 16 m + 8 (matrix % 2) ..
                        const int t = 16 * j + 8 * (ln >> 4) + (ln & 7), ch = 2 * m + ((ln >> 3) & 1);
                        stmatrix_x4_trans(y_base + 64 * t + 16 * (ch ^ ((t >> 1) & 3)), o);
                    }
                }
                __syncwarp();
                // back as rows of the tile, 16 bytes a lane
                {
                    const int t = ln >> 2, ch = ln & 3; // (the swizzle repeats every 8 rows)
                    const unsigned char *src = ytile + 64 * t + 16 * (ch ^ ((t >> 1) & 3));
                    const int left = a.seq - (cb + c) * kDcChunk - kTok * cg - t;
                    const bool in = n0 + row0 + 8 * ch < a.dv; // (dv is a multiple of 8)
#pragma unroll
                    for (int i = 0; i < kTok / 8; ++i)
                        if (in && left > 8 * i)
                            *reinterpret_cast<uint4 *>(yp + i * ystep) = *reinterpret_cast<const uint4 *>(src + 512 * i);
                    yp += (kDcChunk / 8) * ystep;
                }
                if (!kLate) // the next q chunk may land in the tiles' place
                    fence_proxy_async_smem();
            };
            if (outs && !kLate) {
                if (!wait(bar_y, ph)) {
                    ok = false;
                    break;
                }
                emit();
            }
            // ---- H = E_63 H + dH -------------------------------------------------------------
            if (!wait(bar_dh + (kKeys * cg) / 64, ph)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int kb = 0; kb < kKeys / 8; kb += 2) { // 16 keys
                if (kKeys / 16 * cg + kb / 2 < a.nks) {
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t r[8];
                        tmem_ld_frag(lanes + (uint32_t(16 * m) << 16) + kDwH + kKeys * cg + 8 * kb, r);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                H[m][kb + i][x] =
                                    __ffma2_rn(make_float2(em.x, em.x), H[m][kb + i][x], dw_pair(r, 2 * i + x));
                        store_h(m, kb);
                    }
                }
            }
            if (for_m) {
                bool any = false;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int k = 0; k < kKeys / 8; ++k)
                        any = any || H[m][k][0].x != 0.0f || H[m][k][0].y != 0.0f || H[m][k][1].x != 0.0f ||
                              H[m][k][1].y != 0.0f;
                if (any) // (NaN counts)
                    *s_alive = c + 1;
            }
            tmem_st_wait();
            arrive(arr_h);
            if (outs && kLate) {
                if (!wait(bar_y, ph)) {
                    ok = false;
                    break;
                }
                emit();
            }
        }
        if (for_m && ok && tid == 0)
            a.seg_zero[bh * (a.segments - 2) + seg - 1] = zero;
        // where the state goes: N or M, or the final state after the last segment
        float *to = nullptr;
        if (zero)
            ;
        else if (for_m)
            to = a.seg_m + (bh * (a.segments - 2) + seg - 1) * a.dk * a.dk;
        else if (a.pass == 1)
            to = a.seg_n + (bh * (a.segments - 1) + seg) * a.dk * a.dv;
        else if (seg == a.segments - 1 && a.final_state)
            to = a.final_state + bh * a.dk * a.dv;
        if (outs && ok) { // (0 x is 0 for finite x alone)
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int k = 0; k < kKeys / 8; ++k)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        sum = __ffma2_rn(make_float2(0.0f, 0.0f), H[m][k][x], sum);
            if (sum.x != 0.0f || sum.y != 0.0f)
                *s_bad = 1;
        }
        __syncwarp();
        failed = __syncthreads_or(!ok); // before h0's place may take the final state
        if (ok && to && !*s_bad) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int k = 0; k < kKeys / 8; ++k)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (kKeys * cg + 8 * k + tc < a.dk && col + 16 * m + 8 * x < cols) {
                            const int64_t o = sofs + int64_t(8 * k) * cols + 16 * m + 8 * x;
                            to[o] = H[m][k][x].x;
                            to[o + cols] = H[m][k][x].y;
                        }
                    }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tmem, Sh::kCols);
    if (*s_bad && !failed)
        delta_rewalk(a, sm, bh, seg, n0);
}

// ---- the join ------------------------------------------------------------------------
//
// seg_n[s] <- M_s seg_n[s - 1] + seg_n[s] for s = 1 .. segments - 2, in order: the states
// after the segments.  One CTA per head and 16 columns, the running state's columns in
// shared memory, four rows and columns a thread, M staged in blocks ahead of its use; all
// fp32.  32 heads of 128 x 128, 6 segments: 31 us, the latency of the chained products.

constexpr int kDjThreads = 128, kDjCols = 16, kDjK = 32, kDjStages = 3;
constexpr int kDjRow = kDjK + 4; // floats between rows of a staged block of M
constexpr int kDjSmem = (kDjStages * 128 * kDjRow + 128 * kDjCols) * 4;

__global__ void __launch_bounds__(kDjThreads) ss_delta_join_kernel(const DeltaWalkArgs a)
{
    extern __shared__ __align__(16) float dj_sm[];
    float *st = dj_sm + kDjStages * 128 * kDjRow; // [128][kDjCols]
    const int tiles = (a.dv + kDjCols - 1) / kDjCols;
    const int64_t bh = blockIdx.x / unsigned(tiles);
    const int c0 = int(blockIdx.x % unsigned(tiles)) * kDjCols;
    const int row = 4 * (threadIdx.x >> 2), c = 4 * (threadIdx.x & 3);
    const bool in = row < a.dk && c0 + c < a.dv; // (dk and dv are multiples of 8)
    float *n = a.seg_n + bh * (a.segments - 1) * a.dk * a.dv + int64_t(row) * a.dv + c0 + c;
    const float *m = a.seg_m + bh * (a.segments - 2) * a.dk * a.dk;
    const int *zero = a.seg_zero + bh * (a.segments - 2);
    const int64_t nstep = int64_t(a.dk) * a.dv, mstep = int64_t(a.dk) * a.dk;
    // blocks of 128 rows x 32 columns of the M, one after another through three stages
    const int per = (a.dk + kDjK - 1) / kDjK, blocks = (a.segments - 2) * per;
    auto fetch = [&](int i) {
        if (i < blocks && !zero[i / per]) {
            const float *src = m + (i / per) * mstep + (i % per) * kDjK;
            float *dst = dj_sm + (i % kDjStages) * 128 * kDjRow;
#pragma unroll
            for (int u = 0; u < 128 * kDjK / 4 / kDjThreads; ++u) {
                const int e = int(threadIdx.x) + kDjThreads * u, r = e >> 3, k = 4 * (e & 7);
                const bool ok = r < a.dk && (i % per) * kDjK + k < a.dk;
                cp_async16(dst + r * kDjRow + k, ok ? src + int64_t(r) * a.dk + k : m, ok);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    fetch(1);
    float2 acc[4][2];
    auto load_n = [&]() {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (in)
                v = *reinterpret_cast<const float4 *>(n + int64_t(r) * a.dv);
            acc[r][0] = make_float2(v.x, v.y), acc[r][1] = make_float2(v.z, v.w);
        }
    };
    auto keep = [&]() { // the running state's columns
#pragma unroll
        for (int r = 0; r < 4; ++r)
            *reinterpret_cast<float4 *>(st + (row + r) * kDjCols + c) =
                make_float4(acc[r][0].x, acc[r][0].y, acc[r][1].x, acc[r][1].y);
    };
    load_n();
    keep();
    for (int i = 0; i < blocks; ++i) {
        if (i % per == 0) {
            n += nstep;
            load_n();
        }
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads(); // this block has landed, and the one before it has been read
        fetch(i + 2);
        const bool skip = zero[i / per];
        if (!skip) {
            const float *mr = dj_sm + (i % kDjStages) * 128 * kDjRow + row * kDjRow;
            const float *sr = st + (i % per) * kDjK * kDjCols + c;
#pragma unroll
            for (int k = 0; k < kDjK; k += 4) {
                float f[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 v = *reinterpret_cast<const float4 *>(mr + r * kDjRow + k);
                    f[r][0] = v.x, f[r][1] = v.y, f[r][2] = v.z, f[r][3] = v.w;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 v = *reinterpret_cast<const float4 *>(sr + (k + u) * kDjCols);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float2 x = make_float2(f[r][u], f[r][u]);
                        acc[r][0] = __ffma2_rn(x, make_float2(v.x, v.y), acc[r][0]);
                        acc[r][1] = __ffma2_rn(x, make_float2(v.z, v.w), acc[r][1]);
                    }
                }
            }
        }
        if (i % per == per - 1) {
            __syncthreads(); // the state before this segment has been read
            keep();
            if (in && !skip) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<float4 *>(n + int64_t(r) * a.dv) =
                        make_float4(acc[r][0].x, acc[r][0].y, acc[r][1].x, acc[r][1].y);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

} // namespace ss
