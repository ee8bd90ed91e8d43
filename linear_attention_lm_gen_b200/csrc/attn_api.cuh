// Entry points of the softmax-attention operators and the cache operators:
// argument checks, kernel selection and launches. Included by jet_api.cu,
// whose checks and launch helpers it uses.
#pragma once

namespace {

// what jet_attn_rope_append and jet_attn_paged have in common
struct AttnShape {
    int nseq, N, max_pages, n_pages, page_size, Hq, Hk, d;
    jet_dtype dt;
};

constexpr int64_t kMaxTokenStride = 1LL << 32;      // elements between tokens of q, k, v (with N <= 2^24: spans fit)

jet_status check_attn_shape(const AttnShape& a) {
    if (!dtype_ok(a.dt)) return JET_ERR_INVALID_ARG;
    if (a.nseq <= 0 || a.N <= 0 || a.max_pages <= 0 || a.n_pages <= 0 || a.page_size <= 0 || a.Hq <= 0 || a.Hk <= 0 ||
        a.d <= 0 || a.Hq % a.Hk != 0)
        return JET_ERR_INVALID_ARG;
    if (elems({a.N, a.Hq, a.d}) < 0 || elems({a.n_pages, a.page_size, a.Hk, a.d}) < 0) return JET_ERR_INVALID_ARG;
    const bool page_ok = a.page_size >= 16 && a.page_size <= 256 && (a.page_size & (a.page_size - 1)) == 0;
    if (a.d % 16 != 0 || a.d > 128 || !page_ok || a.Hq > 256 || a.Hq / a.Hk > 64 || a.nseq > 65535 ||
        (long long)a.max_pages * a.page_size > 0x40000000LL || a.N > (1 << 24))
        return JET_ERR_UNSUPPORTED;
    return JET_OK;
}

int page_shift_of(int page_size) {
    int sh = 0;
    while ((1 << sh) < page_size) ++sh;
    return sh;
}

// strides of the pools, in elements: rows of d elements that start 16-byte
// aligned and do not overlap their neighbours
jet_status check_pools(const AttnShape& a, const void* k, const void* v, int64_t page_stride, int64_t head_stride,
                       int64_t row_stride) {
    const int64_t align = 16 / (int64_t)esize(a.dt);
    for (int64_t st : {page_stride, head_stride, row_stride}) {
        if (st < a.d || st > (1LL << 38)) return JET_ERR_INVALID_ARG;
        if (st % align != 0) return JET_ERR_MISALIGNED;
    }
    if (elems({a.n_pages, page_stride}) < 0 || elems({a.n_pages, page_stride}) > (1LL << 60)) return JET_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return JET_ERR_MISALIGNED;
    return JET_OK;
}

// bytes from the first to behind the last element of a pool
size_t pool_extent(const AttnShape& a, int64_t page_stride, int64_t head_stride, int64_t row_stride) {
    return esize(a.dt) * (size_t)((a.n_pages - 1) * page_stride + (a.Hk - 1) * head_stride +
                                  (a.page_size - 1) * row_stride + a.d);
}

// N rows of wa elements every sa from a, and of wb every sb from b: an element in common? With one stride exactly, but
// for rows of b before the first or behind the last of a; with two wherever one's extent meets the other's.
bool rows_overlap(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int N, size_t es) {
    if (!overlap(a, es * (size_t)((N - 1) * sa + wa), b, es * (size_t)((N - 1) * sb + wb))) return false;
    if (sa != sb) return true;
    const int64_t S = sa * (int64_t)es, diff = (int64_t)((uintptr_t)b - (uintptr_t)a), r = (diff % S + S) % S;
    return r < wa * (int64_t)es || r + wb * (int64_t)es > S;
}

template <typename T, int LPR, int E, bool INTER>
jet_status launch_append_t(const attn::AppendArgs& a, const attn::Cache& c, const attn::Batch& b, cudaStream_t s) {
    // four tokens to a block once that still fills the GPU several times over
    if (b.N >= 4 * 4 * kMaxSMs)
        return launch(attn::append_kernel<T, 4, LPR, E, INTER>, dim3((b.N + 3) / 4), dim3(attn::APPEND_THREADS), 0, s, a, c,
                      b);
    return launch(attn::append_kernel<T, 1, LPR, E, INTER>, dim3(b.N), dim3(attn::APPEND_THREADS), 0, s, a, c, b);
}
template <typename T, bool INTER>
jet_status launch_append(const attn::AppendArgs& a, const attn::Cache& c, const attn::Batch& b, cudaStream_t s) {
    if (a.rot % 16 == 0)
        return a.d > 64 ? launch_append_t<T, 8, 8, INTER>(a, c, b, s) : launch_append_t<T, 4, 8, INTER>(a, c, b, s);
    return a.d > 64 ? launch_append_t<T, 16, 4, INTER>(a, c, b, s) : launch_append_t<T, 8, 4, INTER>(a, c, b, s);
}

// Workspace of a split attention launch: two slots and a Cut per CTA.
struct SlotLayout {
    size_t ml, cut, bytes;
};
SlotLayout slot_layout(int n_cta, int rows, int d) {
    const size_t o = sizeof(float) * (size_t)n_cta * 2 * rows * d, ml = sizeof(float2) * (size_t)n_cta * 2 * rows;
    return SlotLayout{o, o + ml, o + ml + sizeof(attn::Cut) * (size_t)n_cta};
}
attn::Slots make_slots(void* ws, int n_cta, int rows, int d) {
    uint8_t* p = static_cast<uint8_t*>(ws);
    const SlotLayout L = slot_layout(n_cta, rows, d);
    return attn::Slots{reinterpret_cast<float*>(p), reinterpret_cast<float2*>(p + L.ml),
                       reinterpret_cast<attn::Cut*>(p + L.cut), rows};
}

// tiles of `rows` query rows: whole tokens, or parts of one token's heads
attn::Work make_work(const attn::Cache& c, const attn::Batch& b, int Hk, int G, int window, int rows, int kt, int c0,
                     int min_chunk) {
    const int gt = std::min(G, rows);
    return attn::Work{b, c, Hk, G, window, std::max(1, rows / G), gt, (G + gt - 1) / gt, kt, c0, min_chunk};
}

template <typename T, int RW, int PB, int BLOCKS>
jet_status launch_join(const attn::Work& w, const attn::Slots& sl, void* o, int d, int n_cta, cudaStream_t s) {
    static_assert(4 * kMaxSMs <= attn::MAX_PARTS, "an item's parts");
    const int per = attn::JOIN_WARPS * RW;
    const dim3 grid(n_cta - 1, (sl.rows + per - 1) / per);
    return launch(attn::attn_join_kernel<T, RW, PB, BLOCKS>, grid, dim3(attn::JOIN_WARPS * 32), 0, s, sl, (T*)o, w.Hk * w.G,
                  d, w.gt);
}

template <int DP>
jet_status launch_attn_decode(const void* q, int64_t q_stride, const attn::Cache& c, const attn::Batch& b, void* o,
                              void* ws, int Hk, int G, int d, int window, float scale, cudaStream_t s) {
    typedef attn::DecCfg<DP> C;
    const int n_cta = launch_sms() * C::CTAS;
    // an item's start and end cost a CTA about as much as 192 positions; parts
    // below 128 positions are not worth joining
    const attn::Work w = make_work(c, b, Hk, G, window, attn::DEC_ROWS, attn::DEC_KT, 192, 128);
    const attn::Slots sl = make_slots(ws, n_cta, attn::DEC_ROWS, d);
    auto kern = attn::attn_decode_kernel<DP>;
    if (smem_attr(kern, C::SMEM) != JET_OK) return JET_ERR_CUDA;
    const jet_status st = launch(kern, dim3(n_cta), dim3(attn::DEC_THREADS), C::SMEM, s, (const __nv_bfloat16*)q,
                                 (long long)q_stride, w, sl, (__nv_bfloat16*)o, d, scale * 1.44269504f);
    return st != JET_OK ? st : launch_join<__nv_bfloat16, 1, 16, 2>(w, sl, o, d, n_cta, s);
}

template <int DP>
jet_status launch_attn_f32(const void* q, int64_t q_stride, const attn::Cache& c, const attn::Batch& b, void* o, void* ws,
                           int Hk, int G, int d, int window, float scale, cudaStream_t s) {
    typedef attn::F32Cfg<DP> C;
    const int n_cta = launch_sms() * C::CTAS;
    const attn::Work w = make_work(c, b, Hk, G, window, attn::F32_ROWS, attn::F32_KT, 96, 128);
    const attn::Slots sl = make_slots(ws, n_cta, attn::F32_ROWS, d);
    auto kern = attn::attn_f32_kernel<DP>;
    if (smem_attr(kern, C::SMEM) != JET_OK) return JET_ERR_CUDA;
    const jet_status st = launch(kern, dim3(n_cta), dim3(attn::F32_THREADS), C::SMEM, s,
                                 (const float*)q, (long long)q_stride, w, sl, (float*)o, d, scale * 1.44269504f);
    return st != JET_OK ? st : launch_join<float, 1, 16, 2>(w, sl, o, d, n_cta, s);
}

// pool [n_pages][Hk][page][d] as a 4-D tensor (d, page, Hk, n_pages): a box is 64 columns of up to 128 rows of one page
bool pool_map(CUtensorMap* m, const void* base, const attn::Cache& c, int Hk, int d) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int page = 1 << c.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)page, (cuuint64_t)Hk, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.row_stride * 2, (cuuint64_t)c.head_stride * 2,
                                   (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)std::min(page, attn::CH_KT), 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q [N][Hq][d] as a 3-D tensor (d, Hq, N): a box is 64 columns of the G heads of 128 / G tokens, the rows of one tile
bool query_map(CUtensorMap* m, const void* q, int64_t q_stride, int N, int Hq, int G, int d) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Hq, (cuuint64_t)N};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// query rows of an item: two tiles of whole tokens, at most 128 rows each
int chunk_rows(int G) { return 2 * (128 / G) * G; }

template <int NB>
jet_status launch_attn_chunk(const void* q, int64_t q_stride, const attn::Cache& c, const attn::Batch& b, void* o,
                             void* ws, int Hk, int G, int d, int window, float scale, cudaStream_t s) {
    typedef attn::ChSmem<NB> SM;
    const int n_cta = launch_sms(), rows = chunk_rows(G);
    attn::Work w = make_work(c, b, Hk, G, window, rows, attn::CH_KT, 384, 384);
    w.tpt = 2 * (128 / G);
    const attn::Slots sl = make_slots(ws, n_cta, rows, d);
    CUtensorMap tk, tv, tq;
    if (!pool_map(&tk, c.k, c, Hk, d) || !pool_map(&tv, c.v, c, Hk, d) || !query_map(&tq, q, q_stride, b.N, Hk * G, G, d))
        return JET_ERR_CUDA;
    auto kern = attn::attn_chunk_kernel<NB>;
    if (smem_attr(kern, SM::BYTES) != JET_OK) return JET_ERR_CUDA;
    const jet_status st = launch(kern, dim3(n_cta), dim3(attn::CH_THREADS), SM::BYTES, s, tk, tv, tq, w, sl,
                                 (__nv_bfloat16*)o, d,
                                 scale * 1.44269504f);
    return st != JET_OK ? st : launch_join<__nv_bfloat16, 4, 2, 4>(w, sl, o, d, n_cta, s);
}

// The decode kernel is taken where a sequence's rows fit one of its tiles (one
// read of the cache): 256 sequences of one token 169 us against 209 with the
// chunk kernel. It is also taken where there is little to do at all, since it
// starts sooner: its tiles read the cache again for every 16 rows, so its time
// grows with rows times positions (bounded here by the tables' width or the
// window), and the two are level at about 1.5 million of them, 192 added for
// an item's ends (12 heads over 2; us, decode against chunk kernel: 128 tokens
// over 500 19 / 23, 8 x 8 over 500 16 / 21, 8 x 32 over nothing 11 / 13;
// 8 x 32 over 500 25 / 24, 64 over 3000 26 / 24, 8 x 128 over nothing 28 / 14).
// The bound was fitted on that head shape; at d 64 (16 heads over 8) the decode
// kernel stays ahead longer (4 tokens x 32 over 2000 34 / 57).
//
// Without max_new the average stands for it. That is right for the batches whose
// sequences are alike (2 tokens x 32 over 2000, 12 heads over 2: 28 / 38; 128 x 2
// over 4000, 32 over 8: 326 / 449) and for a piece of 500 tokens among 255 single
// ones over 2000 (10 over 2: 129 / 140), wrong by up to 7 times where such a piece
// has a long cache (over 100000, 10 over 2: 1930 / 257): the caller's to say.
constexpr double kDecodeWork = 1.5e6;
bool take_decode(int nseq, int N, int max_new, long long table_positions, int Hq, int G, int window) {
    const long long typical = max_new > 0 ? max_new : (N + nseq - 1) / nseq;
    if (typical * G <= attn::DEC_ROWS) return true;
    const double seen = window > 0 ? std::min<double>((double)table_positions, (double)window + typical) : (double)table_positions;
    return (double)N * Hq * (seen + 192.0) <= kDecodeWork;
}

}  // namespace

extern "C" {

jet_status jet_attn_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const float* q_gamma, const float* k_gamma, float eps,
                                const float* inv_freq, int rot, int interleaved, void* q_out, int64_t q_out_stride,
                                void* k_pool, void* v_pool, int64_t page_stride, int64_t head_stride,
                                int64_t row_stride, const int* cu_q, const int* kv_lens, const int* page_table,
                                int nseq, int N, int max_pages, int n_pages, int page_size, int Hq, int Hk, int d,
                                jet_dtype dt, void* stream) {
    if (!q || !k || !v || !q_out || !k_pool || !v_pool || !cu_q || !kv_lens || !page_table) return JET_ERR_INVALID_ARG;
    if ((q_gamma == nullptr) != (k_gamma == nullptr)) return JET_ERR_INVALID_ARG;
    const AttnShape a{nseq, N, max_pages, n_pages, page_size, Hq, Hk, d, dt};
    jet_status st = check_attn_shape(a);
    if (st != JET_OK) return st;
    if (rot < 0 || rot > d || (rot > 0 && !inv_freq)) return JET_ERR_INVALID_ARG;
    if (q_gamma && !(eps >= 0.f && eps < INFINITY)) return JET_ERR_INVALID_ARG;
    if (rot % 8 != 0) return JET_ERR_UNSUPPORTED;
    const size_t es = esize(dt);
    for (auto [sd, heads] : {std::pair<int64_t, int>{q_stride, Hq}, {k_stride, Hk}, {v_stride, Hk},
                             {q_out_stride, Hq}}) {
        if (sd < (int64_t)heads * d || sd > kMaxTokenStride) return JET_ERR_INVALID_ARG;
        if (sd % 8 != 0) return JET_ERR_MISALIGNED;
    }
    st = check_pools(a, k_pool, v_pool, page_stride, head_stride, row_stride);
    if (st != JET_OK) return st;
    for (const void* p : {q, k, v, (const void*)q_out})
        if (!aligned16(p)) return JET_ERR_MISALIGNED;
    for (const void* p : {(const void*)q_gamma, (const void*)k_gamma, (const void*)inv_freq, (const void*)cu_q,
                          (const void*)kv_lens, (const void*)page_table})
        if (!aligned_to(p, 4)) return JET_ERR_MISALIGNED;
    auto span = [&](int64_t sd, int heads) { return es * (size_t)((int64_t)(N - 1) * sd + (int64_t)heads * d); };
    // in place over q (same rows, apart from those of k and v), or apart from every input; the pools apart from all of them
    if (q_out == q && q_out_stride == q_stride) {
        for (auto [p, sd] : {std::pair<const void*, int64_t>{k, k_stride}, {v, v_stride}})
            if (rows_overlap(q, q_stride, (int64_t)Hq * d, p, sd, (int64_t)Hk * d, N, es)) return JET_ERR_INVALID_ARG;
    } else {
        for (auto [p, n] : {std::pair<const void*, size_t>{q, span(q_stride, Hq)}, {k, span(k_stride, Hk)},
                            {v, span(v_stride, Hk)}})
            if (overlap(q_out, span(q_out_stride, Hq), p, n)) return JET_ERR_INVALID_ARG;
    }
    const size_t ext = pool_extent(a, page_stride, head_stride, row_stride);
    for (const void* pool : {(const void*)k_pool, (const void*)v_pool})
        for (auto [p, n] : {std::pair<const void*, size_t>{q, span(q_stride, Hq)}, {k, span(k_stride, Hk)},
                            {v, span(v_stride, Hk)}, {q_out, span(q_out_stride, Hq)}})
            if (overlap(pool, ext, p, n)) return JET_ERR_INVALID_ARG;
    if (overlap(k_pool, es * d, v_pool, es * d)) return JET_ERR_INVALID_ARG;       // with the same strides: every row
    const attn::AppendArgs args{q, k, v, q_stride, k_stride, v_stride, q_out_stride, q_gamma, k_gamma, inv_freq, q_out,
                                Hq, Hk, d, rot, eps};
    const attn::Cache c{k_pool, v_pool, page_stride, head_stride, row_stride, page_table, max_pages, n_pages,
                        page_shift_of(page_size)};
    const attn::Batch b{cu_q, kv_lens, nseq, N};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dt == JET_BF16)
        return interleaved ? launch_append<__nv_bfloat16, true>(args, c, b, s)
                           : launch_append<__nv_bfloat16, false>(args, c, b, s);
    return interleaved ? launch_append<float, true>(args, c, b, s) : launch_append<float, false>(args, c, b, s);
}

size_t jet_attn_paged_workspace_size(int nseq, int N, int Hq, int Hk, int d, jet_dtype dt) {
    if (check_attn_shape(AttnShape{nseq, N, 1, 1, 16, Hq, Hk, d, dt}) != JET_OK) return 0;
    if (dt == JET_F32)
        return slot_layout(kMaxSMs * (d <= 64 ? attn::F32Cfg<64>::CTAS : attn::F32Cfg<128>::CTAS), attn::F32_ROWS, d).bytes;
    const int per_sm = d <= 64 ? attn::DecCfg<64>::CTAS : attn::DecCfg<128>::CTAS;
    return std::max(slot_layout(kMaxSMs * per_sm, attn::DEC_ROWS, d).bytes,
                    slot_layout(kMaxSMs, chunk_rows(Hq / Hk), d).bytes);
}

jet_status jet_attn_paged(const void* q, int64_t q_stride, const void* k_pool, const void* v_pool,
                          int64_t page_stride, int64_t head_stride, int64_t row_stride, const int* cu_q,
                          const int* kv_lens, const int* page_table, void* o, void* workspace, size_t ws_bytes,
                          int nseq, int N, int max_new, int max_pages, int n_pages, int page_size, int Hq, int Hk,
                          int d, int window, float scale, jet_dtype dt, void* stream) {
    if (!q || !k_pool || !v_pool || !cu_q || !kv_lens || !page_table || !o) return JET_ERR_INVALID_ARG;
    const AttnShape a{nseq, N, max_pages, n_pages, page_size, Hq, Hk, d, dt};
    jet_status st = check_attn_shape(a);
    if (st != JET_OK) return st;
    if (window < 0 || max_new < 0 || !(scale > 0.f && scale < INFINITY)) return JET_ERR_INVALID_ARG;
    // The axis of the work is measured in 64 bits. Offsets are device data, so every sequence may claim all rows; one
    // costs at most its rows times heads times positions (or rows, if it claims more of them) and a constant below 1024.
    if ((double)nseq * N * Hq * ((double)max_pages * page_size + N + 1024.0) > 0x1p62) return JET_ERR_UNSUPPORTED;
    if (q_stride < (int64_t)Hq * d || q_stride > kMaxTokenStride) return JET_ERR_INVALID_ARG;
    if (q_stride % 8 != 0) return JET_ERR_MISALIGNED;
    st = check_pools(a, k_pool, v_pool, page_stride, head_stride, row_stride);
    if (st != JET_OK) return st;
    for (const void* p : {q, (const void*)o, (const void*)workspace})
        if (!aligned16(p)) return JET_ERR_MISALIGNED;
    for (const int* p : {cu_q, kv_lens, page_table})
        if (!aligned_to(p, 4)) return JET_ERR_MISALIGNED;
    const size_t es = esize(dt), on = es * (size_t)N * Hq * d;
    const size_t qn = es * (size_t)((int64_t)(N - 1) * q_stride + (int64_t)Hq * d);
    const size_t ext = pool_extent(a, page_stride, head_stride, row_stride);
    if (overlap(o, on, q, qn) || overlap(o, on, k_pool, ext) || overlap(o, on, v_pool, ext)) return JET_ERR_INVALID_ARG;
    if (!workspace) ws_bytes = 0;
    if (ws_bytes < jet_attn_paged_workspace_size(nseq, N, Hq, Hk, d, dt)) return JET_ERR_WORKSPACE;
    const attn::Cache c{k_pool, v_pool, page_stride, head_stride, row_stride, page_table, max_pages, n_pages,
                        page_shift_of(page_size)};
    const attn::Batch b{cu_q, kv_lens, nseq, N};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dt == JET_F32)
        return d <= 64 ? launch_attn_f32<64>(q, q_stride, c, b, o, workspace, Hk, Hq / Hk, d, window, scale, s)
                       : launch_attn_f32<128>(q, q_stride, c, b, o, workspace, Hk, Hq / Hk, d, window, scale, s);
    if (!take_decode(nseq, N, max_new, (long long)max_pages * page_size, Hq, Hq / Hk, window))
        return d <= 64 ? launch_attn_chunk<1>(q, q_stride, c, b, o, workspace, Hk, Hq / Hk, d, window, scale, s)
                       : launch_attn_chunk<2>(q, q_stride, c, b, o, workspace, Hk, Hq / Hk, d, window, scale, s);
    return d <= 64 ? launch_attn_decode<64>(q, q_stride, c, b, o, workspace, Hk, Hq / Hk, d, window, scale, s)
                   : launch_attn_decode<128>(q, q_stride, c, b, o, workspace, Hk, Hq / Hk, d, window, scale, s);
}

}  // extern "C"

// ---------------------------------------------------------------- cache operators
namespace {

jet_status make_pools(cache::Pools& P, void* const* pools, const int64_t* entry_bytes, const int64_t* entry_strides,
                      int n_pools, int n_entries) {
    if (!pools || !entry_bytes || !entry_strides || n_pools <= 0 || n_entries <= 0) return JET_ERR_INVALID_ARG;
    if (n_pools > cache::MAX_POOLS) return JET_ERR_UNSUPPORTED;
    P = cache::Pools{};
    P.n = n_pools;
    for (int i = 0; i < n_pools; ++i) {
        if (!pools[i] || entry_bytes[i] <= 0 || entry_strides[i] < entry_bytes[i] || entry_bytes[i] > (1LL << 40) ||
            entry_strides[i] > (1LL << 40))
            return JET_ERR_INVALID_ARG;
        if (!aligned16(pools[i]) || entry_bytes[i] % 16 != 0 || entry_strides[i] % 16 != 0) return JET_ERR_MISALIGNED;
        P.base[i] = static_cast<unsigned char*>(pools[i]);
        P.stride[i] = entry_strides[i];
        P.bytes[i] = entry_bytes[i];
    }
    return JET_OK;
}

// blocks for n entries of every pool: one piece each, up to a limit
unsigned copy_grid(const cache::Pools& P, long long n, long long limit) {
    long long pieces = 0;
    for (int i = 0; i < P.n; ++i) pieces += (P.bytes[i] + cache::PIECE - 1) / cache::PIECE * n;
    return (unsigned)std::max<long long>(1, std::min(pieces, limit));
}

// Every index in range, every destination once and none also a source. One
// bit per entry for each of the two sets; on the stack for the usual pools.
jet_status check_pairs(const int* src, const int* dst, int n, int n_entries) {
    constexpr int kStackWords = 2048;
    uint32_t stack[2 * kStackWords];
    const size_t words = ((size_t)n_entries + 31) / 32;
    uint32_t* mem = stack;
    void* heap = nullptr;
    if (words > kStackWords) {
        heap = std::calloc(2 * words, sizeof(uint32_t));
        if (!heap) return JET_ERR_INVALID_ARG;
        mem = static_cast<uint32_t*>(heap);
    } else {
        std::memset(stack, 0, 2 * words * sizeof(uint32_t));
    }
    uint32_t *is_src = mem, *is_dst = mem + words;
    jet_status st = JET_OK;
    for (int i = 0; i < n && st == JET_OK; ++i) {
        const int a = src[i], b = dst[i];
        if (a < 0 || a >= n_entries || b < 0 || b >= n_entries) { st = JET_ERR_INVALID_ARG; break; }
        if (is_dst[b >> 5] >> (b & 31) & 1u) st = JET_ERR_INVALID_ARG;
        is_src[a >> 5] |= 1u << (a & 31);
        is_dst[b >> 5] |= 1u << (b & 31);
    }
    for (int i = 0; i < n && st == JET_OK; ++i)
        if (is_src[dst[i] >> 5] >> (dst[i] & 31) & 1u) st = JET_ERR_INVALID_ARG;
    std::free(heap);
    return st;
}

template <int CAP>
jet_status launch_copy(const cache::Pools& P, const int* src, const int* dst, int n, cudaStream_t s) {
    cache::Pairs<CAP> pairs;
    for (int i = 0; i < n; ++i) pairs.e[i] = make_int2(src[i], dst[i]);
    return launch(cache::copy_kernel<CAP>, dim3(copy_grid(P, n, 1 << 16)), dim3(cache::THREADS), 0, s, P, pairs, n);
}

constexpr int kFewPairs = 256, kManyPairs = 3584;     // 2 KB and 28 KB of kernel parameters
constexpr int kMaxCompactPages = 1 << 20;
constexpr size_t kPlanSmemMax = kMaxCompactPages / 8; // the plan's bitmap: 128 KB of shared memory

}  // namespace

extern "C" {

jet_status jet_cache_copy(void* const* pools, const int64_t* entry_bytes, const int64_t* entry_strides, int n_pools,
                          int n_entries, const int* src, const int* dst, int n, void* stream) {
    cache::Pools P;
    jet_status st = make_pools(P, pools, entry_bytes, entry_strides, n_pools, n_entries);
    if (st != JET_OK) return st;
    if (n < 0 || (n > 0 && (!src || !dst))) return JET_ERR_INVALID_ARG;
    if (n == 0) return JET_OK;
    st = check_pairs(src, dst, n, n_entries);
    if (st != JET_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int i = 0; i < n && st == JET_OK; i += kManyPairs) {
        const int m = std::min(n - i, kManyPairs);
        st = m <= kFewPairs ? launch_copy<kFewPairs>(P, src + i, dst + i, m, s)
                            : launch_copy<kManyPairs>(P, src + i, dst + i, m, s);
    }
    return st;
}

size_t jet_cache_compact_workspace_size(int n_pages) {
    if (n_pages <= 0 || n_pages > kMaxCompactPages) return 0;
    return 256 + sizeof(int2) * (size_t)((n_pages / 2 + 32) & ~31) + sizeof(int) * (size_t)n_pages;
}

jet_status jet_cache_compact(void* const* pools, const int64_t* entry_bytes, const int64_t* entry_strides,
                             int n_pools, int n_pages, int page_size, const int* page_table, const int* kv_lens,
                             int nseq, int max_pages, int* page_table_out, int* n_live, void* workspace,
                             size_t ws_bytes, void* stream) {
    cache::Pools P;
    jet_status st = make_pools(P, pools, entry_bytes, entry_strides, n_pools, n_pages);
    if (st != JET_OK) return st;
    if (!page_table || !kv_lens || !page_table_out || !n_live || nseq <= 0 || max_pages <= 0 || page_size <= 0)
        return JET_ERR_INVALID_ARG;
    const long long cells = elems({nseq, max_pages});
    if (cells < 0) return JET_ERR_INVALID_ARG;
    if (n_pages > kMaxCompactPages || (page_size & (page_size - 1)) != 0 ||
        (long long)max_pages * page_size > 0x40000000LL)
        return JET_ERR_UNSUPPORTED;
    for (const void* p : {(const void*)page_table, (const void*)kv_lens, (const void*)page_table_out,
                          (const void*)n_live})
        if (!aligned_to(p, 4)) return JET_ERR_MISALIGNED;
    if (!aligned16(workspace)) return JET_ERR_MISALIGNED;
    if (!workspace) ws_bytes = 0;
    if (ws_bytes < jet_cache_compact_workspace_size(n_pages)) return JET_ERR_WORKSPACE;
    const size_t tb = sizeof(int) * (size_t)cells;
    if (page_table_out != page_table && overlap(page_table_out, tb, page_table, tb)) return JET_ERR_INVALID_ARG;
    if (overlap(n_live, 4, page_table, tb) || overlap(n_live, 4, page_table_out, tb) ||
        overlap(n_live, 4, kv_lens, sizeof(int) * (size_t)nseq) ||
        overlap(page_table_out, tb, kv_lens, sizeof(int) * (size_t)nseq))
        return JET_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const size_t moves_bytes = sizeof(int2) * (size_t)((n_pages / 2 + 32) & ~31);
    const cache::PlanOut plan{reinterpret_cast<int*>(w), reinterpret_cast<int2*>(w + 256),
                              reinterpret_cast<int*>(w + 256 + moves_bytes)};
    const int shift = page_shift_of(page_size);
    const size_t smem = sizeof(uint32_t) * (((size_t)n_pages + 31) / 32);
    // The kernel's own variables count against the 48 KB that need no opt-in, so it is asked for from 32 KB on, and
    // always for the largest bitmap: a smaller call on another thread cannot lower it before this one's launch.
    if (smem > 32 * 1024 && smem_attr(cache::compact_plan_kernel, kPlanSmemMax) != JET_OK) return JET_ERR_CUDA;
    st = launch(cache::compact_plan_kernel, dim3(1), dim3(cache::PLAN_THREADS), smem, s, page_table, kv_lens, nseq,
                max_pages, shift, n_pages, plan, n_live);
    if (st != JET_OK) return st;
    // the number of moves is known on the device only: at most half the pages. 16 blocks to an SM, twice what fits at
    // once: 8192 pages half live 186 -> 177 us against 8, and 239 us with a block for every piece there could be
    return launch(cache::compact_move_kernel, dim3(copy_grid(P, std::max(1, n_pages / 2), 16 * kMaxSMs)), dim3(cache::THREADS), 0, s,
                  P, page_table, page_table_out, kv_lens, nseq, max_pages, shift, n_pages, (const int*)n_live, plan);
}

}  // extern "C"
