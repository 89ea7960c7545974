// ss_delta_api.cuh -- host side of the gated delta rule and the group norm: validation,
// dispatch and launch.  Included by ss_api.cu, whose helpers it uses.
#pragma once

namespace {

// Elements from the first to one past the last of `rows` rows of `n` elements, `stride`
// apart; false when that does not fit.
bool row_extent(int64_t rows, int64_t stride, int64_t n, int64_t *out)
{
    int64_t m = 0;
    return stride >= n && mul_ok(rows, stride, &m) && m < INT64_MAX / 8 && ((*out = m - stride + n), true);
}

struct DeltaSizes { // element counts of one call's buffers
    int64_t qn, kn, vn, gates, rows, yn, states;
};

// Everything the two entry points check alike.  rows: batch * seq (prompt) or batch.
int delta_check(int64_t batch, int64_t seq, int64_t heads_k, int64_t heads_v, int64_t dk, int64_t dv, ss_dtype_t dtype,
                const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                const float *g, const float *beta, uint32_t flags, DeltaSizes *z)
{
    if (batch <= 0 || seq <= 0 || heads_k <= 0 || heads_v <= 0 || dk <= 0 || dv <= 0)
        return SS_ERR_SHAPE;
    if (dtype != SS_F32 && dtype != SS_BF16)
        return SS_ERR_DTYPE;
    if (dk > 256 || (flags & ~uint32_t(SS_QK_L2NORM)))
        return SS_ERR_UNSUPPORTED;
    if (heads_v % heads_k != 0 || heads_v > (1 << 20) || dv > (1 << 20))
        return SS_ERR_SHAPE;
    int64_t sh = 0, sd = 0;
    if (!mul_ok(batch, seq, &z->rows) || !mul_ok(z->rows, heads_v, &z->gates) || !mul_ok(z->gates, dv, &z->yn) ||
        !mul_ok(batch, heads_v, &sh) || !mul_ok(sh, dk * dv, &sd) || z->yn > INT64_MAX / 8 || sd > INT64_MAX / 8)
        return SS_ERR_SHAPE;
    z->states = sd;
    if (!row_extent(z->rows, q_stride, heads_k * dk, &z->qn) || !row_extent(z->rows, k_stride, heads_k * dk, &z->kn) ||
        !row_extent(z->rows, v_stride, heads_v * dv, &z->vn))
        return SS_ERR_SHAPE;
    const size_t es = dtype == SS_BF16 ? 2 : 4;
    if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(g, 4) || !aligned(beta, 4))
        return SS_ERR_ALIGN;
    return SS_OK;
}

template <typename T, int R4, int LN> int launch_delta_rec(const ss::DeltaArgs &a, cudaStream_t s)
{
    static std::atomic<uint64_t> smem_done{0};
    constexpr size_t kSmem = ss::DeltaRecSmem<R4, LN>::kBytes;
    const int st = ensure_smem(ss::ss_delta_rec_kernel<T, R4, LN>, kSmem, smem_done);
    if (st != SS_OK)
        return st;
    const int64_t tiles = (a.dv + ss::dr_cols(LN) - 1) / ss::dr_cols(LN);
    int64_t grid = 0;
    if (!mul_ok(a.batch * a.heads_v, tiles, &grid) || grid > 0x7fffffffLL)
        return SS_ERR_SHAPE;
    ss::ss_delta_rec_kernel<T, R4, LN><<<unsigned(grid), ss::dr_threads(LN), kSmem, s>>>(a);
    return launch_status();
}

// Four columns a CTA (16 lanes each) where all CTAs then run at once, sixteen (8 lanes) where
// they would not: 300 tokens x 4 heads of 128, 34 us against 48 us; 2 heads of 256, 45 us
// against 86 us.
template <typename T> int dispatch_delta_rec(const ss::DeltaArgs &a, cudaStream_t s)
{
    int sms = 0;
    if (device_sm_count(&sms) != SS_OK)
        return SS_ERR_CUDA;
    const int64_t heads = a.batch * a.heads_v, tiles = (a.dv + ss::dr_cols(16) - 1) / ss::dr_cols(16);
    if (heads <= sms && heads * tiles <= sms) {
        if (a.dk <= 64)
            return launch_delta_rec<T, 2, 16>(a, s);
        return a.dk <= 128 ? launch_delta_rec<T, 4, 16>(a, s) : launch_delta_rec<T, 8, 16>(a, s);
    }
    if (a.dk <= 32)
        return launch_delta_rec<T, 1, 8>(a, s);
    if (a.dk <= 64)
        return launch_delta_rec<T, 2, 8>(a, s);
    return a.dk <= 128 ? launch_delta_rec<T, 4, 8>(a, s) : launch_delta_rec<T, 8, 8>(a, s);
}

// ---- the chunked form ----------------------------------------------------------------

// Shapes the chunked form takes (bf16; q, k and v as rows of whole 16-byte vectors, which
// TMA asks for; keys of 8 would leave seven eighths of the tiles empty).  Prompts of up to
// 16 tokens are walked token by token.  The state then keeps float32's accuracy where a prompt
// comes in many small pieces (the chunked form costs it 5e-6 a call), and with few heads it is
// the faster form, too: 16 heads x 16 tokens 14 us against 22 us, 32 heads 22 us in either.
// With many heads it is the slower one at any length: 256 heads x 16 tokens 113 us against
// 31 us, 2048 heads 782 us against 137 us.
bool delta_chunked_shape(int64_t batch, int64_t seq, int64_t dk, int64_t dv, ss_dtype_t dtype)
{
    return dtype == SS_BF16 && dk >= 16 && dk <= 128 && dk % 8 == 0 && dv % 8 == 0 && seq > 16 && seq < (int64_t(1) << 31) - 64 &&
           batch < (int64_t(1) << 31);
}

// Segments of the two-pass walk (1: one pass): as many as make 192 walks in pass 2, each of 12
// chunks or more.  Two passes and the join against one pass, heads of 128 x 128, in us:
//   heads            1          8         16         32         48         64
//   36 chunks   98 / 123  102 / 127  107 / 131  121 / 141  135 / 152  186 / 162
//   64 chunks  115 / 207  121 / 213  131 / 223  197 / 238  234 / 254  291 / 268
//   256 chunks 188 / 766  262 / 817  362 / 846  537 / 893  756 / 944  983 / 1002
// (64 heads of 36 to 64 chunks are on the wrong side by up to 15%.)  With 148 walks, one an SM:
// 573 us for 256 chunks x 32 heads, but 242, 317 and 694 us with 8, 16 and 48 heads.  Segments
// of 8 chunks and more: 88 us for 36 chunks of one head, but 217 us for 256, whose join is
// longer; of 16 and more: 131 us for 256 chunks of one head, none for 36.
constexpr int64_t kDeltaWalks = 192; // of pass 2
int64_t delta_segments(int64_t heads, int64_t tiles, int64_t chunks)
{
    int64_t segs = heads > kDeltaWalks ? 1 : kDeltaWalks / (heads * tiles);
    segs = segs < chunks / 12 ? segs : chunks / 12;
    return segs < 3 ? 1 : segs;
}

bool delta_chunked(const ss::DeltaArgs &a, const void *workspace)
{
    return workspace && delta_chunked_shape(a.batch, a.seq, a.dk, a.dv, SS_BF16) && aligned(a.q, 16) &&
           aligned(a.k, 16) && aligned(a.v, 16) && aligned(a.y, 16) && a.q_stride % 8 == 0 && a.k_stride % 8 == 0 && a.v_stride % 8 == 0 &&
           a.q_stride * a.seq < (int64_t(1) << 38) && a.k_stride * a.seq < (int64_t(1) << 38) &&
           a.v_stride * a.seq < (int64_t(1) << 38) &&
           int64_t(a.heads_v) * a.dv * a.seq < (int64_t(1) << 38); // (byte strides of a tensor map end at 2^40)
}

// 4-D map (d, head, token, batch) over rows of heads, box (64, 1, 64 tokens, 1),
// 128-byte swizzle.
bool encode_heads(CUtensorMap *map, const void *base, int64_t d, int64_t heads, int64_t seq, int64_t batch,
                  int64_t stride)
{
    PFN_cuTensorMapEncodeTiled enc = tensor_map_encoder();
    if (!enc)
        return false;
    const cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(seq), cuuint64_t(batch)};
    const cuuint64_t strides[3] = {cuuint64_t(d) * 2, cuuint64_t(stride) * 2, cuuint64_t(stride) * 2 * cuuint64_t(seq)};
    const cuuint32_t box[4] = {64, 1, uint32_t(ss::kDcChunk), 1}, estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G>
int launch_delta_walk_t(const ss::DeltaWalkArgs &w, const ss::DeltaWalkMaps &maps, unsigned grid, uint32_t *status,
                        cudaStream_t s)
{
    static std::atomic<uint64_t> smem_done{0};
    const int st = ensure_smem(ss::ss_delta_walk_kernel<G>, size_t(ss::DwSmem<G>::kBytes), smem_done);
    if (st != SS_OK)
        return st;
    ss::ss_delta_walk_kernel<G><<<grid, ss::DwShape<G>::kThreads, ss::DwSmem<G>::kBytes, s>>>(w, maps, status);
    return launch_status();
}

// Up to one walk per SM: sixteen compute warps each; more: two CTAs of eight per SM.
int launch_delta_walk(const ss::DeltaWalkArgs &w, const ss::DeltaWalkMaps &maps, int64_t grid, uint32_t *status,
                      cudaStream_t s)
{
    int sms = 0;
    if (device_sm_count(&sms) != SS_OK)
        return SS_ERR_CUDA;
    if (grid > 0x7fffffffLL)
        return SS_ERR_SHAPE;
    return grid <= sms ? launch_delta_walk_t<4>(w, maps, unsigned(grid), status, s)
                       : launch_delta_walk_t<2>(w, maps, unsigned(grid), status, s);
}

int launch_delta_chunked(const ss::DeltaArgs &a, void *workspace, cudaStream_t s)
{
    static std::atomic<uint64_t> smem_done{0};
    int st = ensure_smem(ss::ss_delta_prep_kernel, size_t(ss::DeltaPrepSmem::kBytes), smem_done);
    if (st != SS_OK)
        return st;
    uint32_t *status = nullptr;
    if (status_word_address(&status) != SS_OK)
        return SS_ERR_CUDA;
    ss::DeltaPrepArgs p{};
    p.d = a;
    p.nchunks = int((a.seq + ss::kDcChunk - 1) / ss::kDcChunk);
    p.blocks = static_cast<unsigned char *>(workspace);
    ss::DeltaWalkArgs w{};
    w.d = a;
    w.batch = a.batch;
    w.seq = int(a.seq);
    w.heads_v = a.heads_v;
    w.ratio = a.ratio;
    w.dk = a.dk;
    w.dv = a.dv;
    w.nchunks = p.nchunks;
    w.col_tiles = (a.dv + 127) / 128;
    w.nks = (a.dk + 15) / 16;
    w.blocks = p.blocks;
    const int64_t segs = delta_segments(a.batch * a.heads_v, w.col_tiles, p.nchunks);
    w.seg_chunks = int((p.nchunks + segs - 1) / segs);
    w.segments = (p.nchunks + w.seg_chunks - 1) / w.seg_chunks;
    w.seg_n = reinterpret_cast<float *>(p.blocks + a.batch * a.heads_v * p.nchunks * ss::kDcBlockBytes);
    w.seg_m = w.seg_n + a.batch * a.heads_v * (w.segments - 1) * a.dk * a.dv;
    float *end_m = w.seg_m + a.batch * a.heads_v * (w.segments - 2) * a.dk * a.dk;
    w.seg_h0 = a.h0 && a.final_state == a.h0 ? end_m : nullptr;
    w.seg_zero = reinterpret_cast<int *>(end_m + a.batch * a.heads_v * a.dk * a.dv);
    w.hold = g_gated_path.load(std::memory_order_relaxed) == 3 ? 1 : 0;
    w.h0 = a.h0;
    w.g = a.g;
    w.reset = a.reset;
    w.y = static_cast<__nv_bfloat16 *>(a.y);
    w.final_state = a.final_state;
    int64_t units = 0, grid = 0;
    if (!mul_ok(a.batch * a.heads_v, p.nchunks, &units) || units > 0x7fffffffLL ||
        !mul_ok(a.batch * a.heads_v, w.col_tiles, &grid) || grid > 0x7fffffffLL)
        return SS_ERR_SHAPE;
    ss::DeltaWalkMaps maps;
    memset(&maps, 0, sizeof(maps));
    if (!encode_heads(&maps.q, a.q, a.dk, a.heads_k, a.seq, a.batch, a.q_stride) ||
        !encode_heads(&maps.k, a.k, a.dk, a.heads_k, a.seq, a.batch, a.k_stride) ||
        !encode_heads(&maps.v, a.v, a.dv, a.heads_v, a.seq, a.batch, a.v_stride))
        return SS_ERR_CUDA;
    ss::ss_delta_prep_kernel<<<unsigned(units), ss::kDpThreads, ss::DeltaPrepSmem::kBytes, s>>>(p);
    if ((st = launch_status()) != SS_OK)
        return st;
    if (w.segments == 1)
        return launch_delta_walk(w, maps, grid, status, s);
    const int64_t heads = a.batch * a.heads_v;
    w.pass = 1;
    st = launch_delta_walk(w, maps, heads * (w.col_tiles + (w.segments - 2) * (w.col_tiles + 1)), status, s);
    if (st != SS_OK)
        return st;
    static std::atomic<uint64_t> join_done{0};
    if ((st = ensure_smem(ss::ss_delta_join_kernel, size_t(ss::kDjSmem), join_done)) != SS_OK)
        return st;
    ss::ss_delta_join_kernel<<<unsigned(heads * ((a.dv + ss::kDjCols - 1) / ss::kDjCols)), ss::kDjThreads, ss::kDjSmem,
                               s>>>(w);
    if ((st = launch_status()) != SS_OK)
        return st;
    w.pass = 2;
    return launch_delta_walk(w, maps, heads * w.col_tiles * w.segments, status, s);
}

template <typename T, int J> int launch_delta_update(ss::DeltaUpdateArgs a, cudaStream_t s)
{
    a.col_tiles = (a.dv + ss::kDuCols - 1) / ss::kDuCols;
    int64_t grid = 0;
    if (!mul_ok(a.batch * a.heads_v, a.col_tiles, &grid) || grid > 0x7fffffffLL)
        return SS_ERR_SHAPE;
    const bool vec = a.dv % 4 == 0 && aligned(a.state, 16);
    if (vec && a.dk == 16 * J && a.dv % ss::kDuCols == 0)
        ss::ss_delta_update_kernel<T, J, true, true><<<unsigned(grid), ss::kDuThreads, 0, s>>>(a);
    else if (vec)
        ss::ss_delta_update_kernel<T, J, true, false><<<unsigned(grid), ss::kDuThreads, 0, s>>>(a);
    else
        ss::ss_delta_update_kernel<T, J, false, false><<<unsigned(grid), ss::kDuThreads, 0, s>>>(a);
    return launch_status();
}

template <typename T> int dispatch_delta_update(const ss::DeltaUpdateArgs &a, cudaStream_t s)
{
    if (a.dk <= 64)
        return launch_delta_update<T, 4>(a, s);
    return a.dk <= 128 ? launch_delta_update<T, 8>(a, s) : launch_delta_update<T, 16>(a, s);
}

template <typename T, int VEC, int NV, bool CTA> int launch_group_norm(const ss::GroupNormArgs &a, cudaStream_t s)
{
    int sms = 0;
    if (device_sm_count(&sms) != SS_OK)
        return SS_ERR_CUDA;
    const int64_t per_cta = CTA ? 1 : ss::kGnThreads >> a.team_log2;
    const int64_t blocks = (a.rows * a.groups + per_cta - 1) / per_cta;
    const int64_t most = int64_t(sms) * 16;
    const unsigned grid = unsigned(blocks < most ? blocks : most);
    if (VEC > 1 && a.size == (CTA ? ss::kGnThreads : 1 << a.team_log2) * VEC * NV)
        ss::ss_group_norm_kernel<T, VEC, NV, CTA, (VEC > 1)><<<grid, ss::kGnThreads, 0, s>>>(a);
    else
        ss::ss_group_norm_kernel<T, VEC, NV, CTA, false><<<grid, ss::kGnThreads, 0, s>>>(a);
    return launch_status();
}

// Teams: the fewest lanes of a warp that hold a group in `kMost` vectors each, or a warp
// with up to eight; beyond that the CTA.  kMost 2 for 16-byte vectors (16384 x 32 groups
// of 128 bf16 with a gate, guarded: 72 us against 78-90 with one vector a lane; unguarded
// 70 us), 8 for single elements (16384 x 5 groups of 83: 27 us against 31 with a whole warp).
template <typename T, int VEC> int dispatch_group_norm(ss::GroupNormArgs &a, cudaStream_t s)
{
    constexpr int kMost = VEC == 1 ? 8 : 2;
    const int vecs = (a.size + VEC - 1) / VEC;
    a.team_log2 = 0;
    while (a.team_log2 < 5 && (kMost << a.team_log2) < vecs)
        ++a.team_log2;
    switch ((vecs + (1 << a.team_log2) - 1) >> a.team_log2) {
    case 1: return launch_group_norm<T, VEC, 1, false>(a, s);
    case 2: return launch_group_norm<T, VEC, 2, false>(a, s);
    case 3: return launch_group_norm<T, VEC, 3, false>(a, s);
    case 4: return launch_group_norm<T, VEC, 4, false>(a, s);
    case 5: return launch_group_norm<T, VEC, 5, false>(a, s);
    case 6: return launch_group_norm<T, VEC, 6, false>(a, s);
    case 7:
    case 8: return launch_group_norm<T, VEC, 8, false>(a, s);
    }
    if (vecs <= 4 * ss::kGnThreads)
        return launch_group_norm<T, VEC, 4, true>(a, s);
    if constexpr (VEC == 1) {
        if (vecs > 16 * ss::kGnThreads)
            return launch_group_norm<T, VEC, 64, true>(a, s);
    }
    return launch_group_norm<T, VEC, VEC == 8 ? 8 : 16, true>(a, s);
}

} // namespace

extern "C" {

int ss_delta_scan(int64_t batch, int64_t seq, int64_t heads_k, int64_t heads_v, int64_t dk, int64_t dv,
                  ss_dtype_t dtype, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                  int64_t v_stride, const float *g, const float *beta, const uint8_t *reset, const float *h0,
                  float scale, uint32_t flags, void *outputs, float *final_state, void *workspace,
                  size_t workspace_bytes, ss_stream_t stream)
{
    if (!q || !k || !v || !outputs)
        return SS_ERR_NULL;
    DeltaSizes z{};
    const int st = delta_check(batch, seq, heads_k, heads_v, dk, dv, dtype, q, q_stride, k, k_stride, v, v_stride, g,
                               beta, flags, &z);
    if (st != SS_OK)
        return st;
    const size_t es = dtype == SS_BF16 ? 2 : 4;
    if (!aligned(outputs, es) || !aligned(h0, 4) || !aligned(final_state, 4) || !aligned(workspace, 16))
        return SS_ERR_ALIGN;
    if (workspace && int64_t(workspace_bytes) < ss_delta_workspace_bytes(batch, seq, heads_k, heads_v, dk, dv, dtype))
        return SS_ERR_WORKSPACE;
    const size_t ybytes = size_t(z.yn) * es, sbytes = size_t(z.states) * 4;
    const void *in_p[] = {q, k, v, g, beta, reset, h0};
    const size_t in_n[] = {size_t(z.qn) * es, size_t(z.kn) * es, size_t(z.vn) * es, size_t(z.gates) * 4,
                           size_t(z.gates) * 4, size_t(z.rows), sbytes};
    const void *out_p[] = {outputs, final_state, workspace};
    const size_t out_n[] = {ybytes, sbytes, workspace_bytes};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 7; ++i) {
            if (o == 1 && i == 6 && final_state == h0)
                continue; // chaining in place
            if (overlaps(out_p[o], out_n[o], in_p[i], in_n[i]))
                return SS_ERR_ALIAS;
        }
        for (int i = 0; i < o; ++i)
            if (overlaps(out_p[o], out_n[o], out_p[i], out_n[i]))
                return SS_ERR_ALIAS;
    }
    ss::DeltaArgs a{};
    a.batch = batch;
    a.seq = seq;
    a.heads_k = int(heads_k);
    a.heads_v = int(heads_v);
    a.ratio = int(heads_v / heads_k);
    a.dk = int(dk);
    a.dv = int(dv);
    a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.g = g;
    a.beta = beta;
    a.reset = reset;
    a.h0 = h0;
    a.y = outputs;
    a.final_state = final_state;
    a.scale = scale;
    a.l2norm = (flags & SS_QK_L2NORM) ? 1 : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == SS_F32)
        return dispatch_delta_rec<float>(a, s);
    return delta_chunked(a, workspace) ? launch_delta_chunked(a, workspace, s) : dispatch_delta_rec<__nv_bfloat16>(a, s);
}

int64_t ss_delta_workspace_bytes(int64_t batch, int64_t seq, int64_t heads_k, int64_t heads_v, int64_t dk, int64_t dv,
                                 ss_dtype_t dtype)
{
    if (batch <= 0 || seq <= 0 || heads_k <= 0 || heads_v <= 0 || dk <= 0 || dv <= 0 || heads_v % heads_k ||
        !delta_chunked_shape(batch, seq, dk, dv, dtype))
        return 0;
    int64_t heads = 0, n = 0;
    const int64_t chunks = (seq + ss::kDcChunk - 1) / ss::kDcChunk;
    if (!mul_ok(batch, heads_v, &heads) || !mul_ok(heads, chunks, &n) || !mul_ok(n, ss::kDcBlockBytes, &n))
        return 0;
    // the states of the segments, when the sequence is cut (few heads: they are small)
    const int64_t segs = delta_segments(heads, (dv + 127) / 128, chunks);
    return segs == 1 ? n : n + heads * 4 * (dk * (segs * dv + (segs - 2) * dk) + (segs - 2));
}

int ss_delta_update(int64_t batch, int64_t heads_k, int64_t heads_v, int64_t dk, int64_t dv, ss_dtype_t dtype,
                    float *state, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                    int64_t v_stride, const float *g, const float *beta, float scale, uint32_t flags, void *y,
                    ss_stream_t stream)
{
    if (!state || !q || !k || !v || !y)
        return SS_ERR_NULL;
    DeltaSizes z{};
    const int st = delta_check(batch, 1, heads_k, heads_v, dk, dv, dtype, q, q_stride, k, k_stride, v, v_stride, g,
                               beta, flags, &z);
    if (st != SS_OK)
        return st;
    const size_t es = dtype == SS_BF16 ? 2 : 4;
    if (!aligned(y, es) || !aligned(state, 4))
        return SS_ERR_ALIGN;
    const size_t ybytes = size_t(z.yn) * es, sbytes = size_t(z.states) * 4;
    const void *in_p[] = {q, k, v, g, beta};
    const size_t in_n[] = {size_t(z.qn) * es, size_t(z.kn) * es, size_t(z.vn) * es, size_t(z.gates) * 4,
                           size_t(z.gates) * 4};
    for (int i = 0; i < 5; ++i)
        if (overlaps(y, ybytes, in_p[i], in_n[i]) || overlaps(state, sbytes, in_p[i], in_n[i]))
            return SS_ERR_ALIAS;
    if (overlaps(y, ybytes, state, sbytes))
        return SS_ERR_ALIAS;
    ss::DeltaUpdateArgs a{};
    a.batch = batch;
    a.heads_k = int(heads_k);
    a.heads_v = int(heads_v);
    a.ratio = int(heads_v / heads_k);
    a.dk = int(dk);
    a.dv = int(dv);
    a.state = state;
    a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.g = g;
    a.beta = beta;
    a.y = y;
    a.scale = scale;
    a.l2norm = (flags & SS_QK_L2NORM) ? 1 : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == SS_BF16 ? dispatch_delta_update<__nv_bfloat16>(a, s) : dispatch_delta_update<float>(a, s);
}

int ss_group_norm(int64_t rows, int64_t groups, int64_t size, ss_dtype_t dtype, const void *x, int64_t x_stride,
                  const void *gate, int64_t gate_stride, const float *weight, const float *bias, float eps,
                  uint32_t flags, void *y, ss_stream_t stream)
{
    if (!x || !y)
        return SS_ERR_NULL;
    if (rows <= 0 || groups <= 0 || size <= 0)
        return SS_ERR_SHAPE;
    if (dtype != SS_F32 && dtype != SS_BF16)
        return SS_ERR_DTYPE;
    if (size > SS_GROUP_NORM_MAX_SIZE ||
        (flags & ~uint32_t(SS_NORM_CENTER | SS_NORM_GATE_FIRST | SS_NORM_SILU | SS_NORM_SHARED)))
        return SS_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f))
        return SS_ERR_UNSUPPORTED;
    int64_t ch = 0, yn = 0, xn = 0, zn = 0, items = 0;
    if (!mul_ok(groups, size, &ch) || ch > 0x7fffffffLL || !mul_ok(rows, groups, &items) || !mul_ok(rows, ch, &yn) ||
        yn > INT64_MAX / 8 || !row_extent(rows, x_stride, ch, &xn) || (gate && !row_extent(rows, gate_stride, ch, &zn)))
        return SS_ERR_SHAPE;
    const size_t es = dtype == SS_BF16 ? 2 : 4;
    if (!aligned(x, es) || !aligned(gate, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(bias, 4))
        return SS_ERR_ALIGN;
    const size_t pn = size_t((flags & SS_NORM_SHARED) ? size : ch) * 4;
    const void *in_p[] = {x, gate, weight, bias};
    const size_t in_n[] = {size_t(xn) * es, size_t(zn) * es, pn, pn};
    for (int i = 0; i < 4; ++i)
        if (overlaps(y, size_t(yn) * es, in_p[i], in_n[i]))
            return SS_ERR_ALIAS;
    ss::GroupNormArgs a{};
    a.rows = rows;
    a.groups = int(groups);
    a.size = int(size);
    a.x = x;
    a.gate = gate;
    a.x_stride = x_stride;
    a.gate_stride = gate_stride;
    a.weight = weight;
    a.bias = bias;
    a.y = y;
    a.eps = eps;
    a.inv_size = 1.0f / float(size);
    a.mode = int(flags);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t per = 16 / int64_t(es);
    const bool vec = size % per == 0 && aligned(x, 16) && x_stride % per == 0 && aligned(y, 16) &&
                     (!gate || (aligned(gate, 16) && gate_stride % per == 0)) && aligned(weight, 16) &&
                     aligned(bias, 16);
    if (dtype == SS_BF16)
        return vec ? dispatch_group_norm<__nv_bfloat16, 8>(a, s) : dispatch_group_norm<__nv_bfloat16, 1>(a, s);
    return vec ? dispatch_group_norm<float, 4>(a, s) : dispatch_group_norm<float, 1>(a, s);
}

} // extern "C"
