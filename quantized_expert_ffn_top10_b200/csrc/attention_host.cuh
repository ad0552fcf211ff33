// Host side of the attention half of a layer: argument checks, workspace layout
// and launches of the kernels in kvcache.cuh and attention.cuh.  Part of
// libmoe.cu's translation unit.
#pragma once

#include <math.h>

namespace {

int check_kv_desc(const moe_kv_desc* d) {
    if (!d || !d->k_cache || !d->v_cache) return MOE_ERR_ARG;
    if (d->reserved[0] || d->reserved[1]) return MOE_ERR_SHAPE;
    if (d->kv_type != MOE_KV_BF16 && d->kv_type != MOE_KV_E4M3) return MOE_ERR_SHAPE;
    if (d->head_dim != 64 && d->head_dim != 128) return MOE_ERR_SHAPE;
    if (d->n_kv_heads < 1 || d->n_heads < 1 || d->n_heads > MOE_ATTN_MAX_HEADS || d->n_heads % d->n_kv_heads)
        return MOE_ERR_SHAPE;
    if (d->n_pages < 1 || d->page_size < 1 || (int64_t)d->n_pages * d->page_size > 0x7fffffffLL) return MOE_ERR_RANGE;
    const int64_t per16 = d->kv_type == MOE_KV_BF16 ? 8 : 16;  // elements in 16 bytes
    for (const int64_t s : {d->page_stride, d->token_stride, d->head_stride})
        if (s < 0 || s % per16) return MOE_ERR_SHAPE;
    if (!aligned(d->k_cache, 16) || !aligned(d->v_cache, 16)) return MOE_ERR_ARG;
    if (!aligned(d->k_scale, 4) || !aligned(d->v_scale, 4)) return MOE_ERR_ARG;
    if (d->kv_type == MOE_KV_BF16 && (d->k_scale || d->v_scale)) return MOE_ERR_ARG;
    return MOE_OK;
}

inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && n && m && a < b + m && b < a + n;
}

// Whether T rows of w elements, s apart, and T rows of v elements, r apart, share memory.  Rows of equal strides may
// interleave (parts of one projection buffer); unequal ones may not meet at all.
inline bool rows_overlap(const uint16_t* p, int64_t s, int64_t w, const uint16_t* q, int64_t r, int64_t v, int T) {
    if (!overlap(p, ((size_t)(T - 1) * s + w) * 2, q, ((size_t)(T - 1) * r + v) * 2)) return false;
    if (s != r) return true;
    const int64_t at = ((q - p) % s + s) % s;  // where q's rows start in p's
    return at < w || at + v > s;
}

// Four tokens a CTA once that still leaves four CTAs for every SM; below, one token a CTA for the latency.
template <int D, bool F8>
void launch_rope(const RopeArgs& a, cudaStream_t st) {
    const int tok = a.T >= QR_TOKENS * 4 * 148 ? QR_TOKENS : 1, pieces = tok * (a.Hq + 2 * a.Hk) * (D / 16);
    const int each = tok == 1 ? 1 : QR_UNROLL;  // pieces a thread
    const int threads = std::min(qr_threads(F8, tok), std::max(64, ((pieces + each - 1) / each + 31) / 32 * 32));
    if (tok == 1) k_qk_norm_rope<D, F8, 1><<<a.T, threads, 0, st>>>(a);
    else k_qk_norm_rope<D, F8, QR_TOKENS><<<(a.T + tok - 1) / tok, threads, 0, st>>>(a);
}

// ---------------------------------------------------------------- attention

struct AttnWs {
    size_t hdr, ml, part, total;
};

AttnWs attn_ws(int D) {
    AttnWs w{};
    size_t o = 0;
    auto put = [&](size_t bytes) { size_t r = o; o += al(bytes); return r; };
    const size_t slots = (size_t)2 * ATT_MAX_SMS * ATT_PART_ROWS;  // two per CTA, rows of the widest kernel
    w.hdr = put(ATT_MAX_SMS * ATT_MAX_PER_SM * sizeof(int4));
    w.ml = put(slots * sizeof(float2));
    w.part = put(slots * D * 4);
    w.total = o;
    return w;
}

struct AttnCall {
    const moe_kv_desc* d;
    const uint16_t* q;
    int64_t q_stride;
    int T, B;
    const int32_t *cu, *kv_len, *table;
    int width, max_q;
    float scale, softcap;
    int window;
    const float* slopes;
    const int32_t* prefix;
    uint16_t* out;
    float* lse;
    uint8_t* ws;
    size_t ws_bytes;
    cudaStream_t st;
};

int check_attn(const AttnCall& c, int max_T) {
    int rc = check_kv_desc(c.d);
    if (rc) return rc;
    if (c.T < 0 || c.T > max_T || c.B < 0 || c.B > MOE_ATTN_MAX_B || c.width < 1 || c.max_q < 1) return MOE_ERR_RANGE;
    if (c.window < 0 || !isfinite(c.softcap) || !isfinite(c.scale)) return MOE_ERR_RANGE;
    if (c.softcap != 0.f && !(c.softcap >= 1e-30f)) return MOE_ERR_RANGE;  // (its reciprocal is used)
    const int64_t row = (int64_t)c.d->n_heads * c.d->head_dim;
    if (c.q_stride < row || c.q_stride % 8) return MOE_ERR_SHAPE;
    if (c.T == 0 || c.B == 0) return MOE_OK;  // nothing to do: the buffers may be null
    if (!c.q || !c.cu || !c.kv_len || !c.table || !c.out || !c.ws) return MOE_ERR_ARG;
    if (!aligned(c.q, 16) || !aligned(c.out, 16) || !aligned(c.ws, kAlign)) return MOE_ERR_ARG;
    for (const void* p : {(const void*)c.cu, (const void*)c.kv_len, (const void*)c.table, (const void*)c.slopes,
                          (const void*)c.prefix, (const void*)c.lse})
        if (!aligned(p, 4)) return MOE_ERR_ARG;
    if (overlap(c.q, ((size_t)(c.T - 1) * c.q_stride + row) * 2, c.out, (size_t)c.T * row * 2)) return MOE_ERR_ARG;
    if (c.ws_bytes < attn_ws(c.d->head_dim).total) return MOE_ERR_WS;
    return MOE_OK;
}

int g_attn_sms[256];  // SMs per device once its kernels are set up (0 = not yet)

template <int D, bool F8>
cudaError_t attn_attrs() {
    cudaError_t e = set_smem(k_attn_rows<D, F8, 1, 1, 4>, AttCfg<D, F8, 1, 1, 4>::SMEM);
    if (e == cudaSuccess) e = set_smem(k_attn_rows<D, F8, 2, 1, 4>, AttCfg<D, F8, 2, 1, 4>::SMEM);
    if (e == cudaSuccess) e = set_smem(k_attn_rows<D, F8, 2, 2, 2>, AttCfg<D, F8, 2, 2, 2>::SMEM);
    if (e == cudaSuccess) e = set_smem(k_attn_rows<D, F8, 2, 4, 2>, AttCfg<D, F8, 2, 4, 2>::SMEM);
    if (e == cudaSuccess) e = set_smem(k_attn_chunk<D, F8, 0>, AcCfg<D, F8>::SMEM);
    if (e == cudaSuccess) e = set_smem(k_attn_chunk<D, F8, 1>, AcCfg<D, F8>::SMEM);
    if (e == cudaSuccess) e = set_smem(k_attn_chunk<D, F8, 2>, AcCfg<D, F8>::SMEM);
    if (e == cudaSuccess) e = set_smem(k_attn_chunk<D, F8, 3>, AcCfg<D, F8>::SMEM);
    return e;
}

int attn_init(int* sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return MOE_ERR_CUDA;
    std::lock_guard<std::mutex> g(g_mu);
    if (!g_attn_sms[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return MOE_ERR_CUDA;
        if (attn_attrs<64, false>() != cudaSuccess || attn_attrs<64, true>() != cudaSuccess ||
            attn_attrs<128, false>() != cudaSuccess || attn_attrs<128, true>() != cudaSuccess)
            return MOE_ERR_CUDA;
        g_attn_sms[dev] = n;
    }
    *sms = g_attn_sms[dev];
    return MOE_OK;
}

// A cache as a 4-D tensor (element, token, head, page); a box is min(page, 128)
// tokens of one head of one page, 64 bf16 columns with the 128-byte swizzle or a
// whole e4m3 row without one.  False for pages that such boxes do not tile.
template <int D, bool F8>
bool tmap_cache(CUtensorMap* m, const uint8_t* base, const AttnArgs& a) {
    const int ps = a.page_size;
    if (ps < 8 || (ps & (ps - 1)) || !encoder()) return false;
    cuuint64_t dims[4] = {D, (cuuint64_t)ps, (cuuint64_t)a.Hk, (cuuint64_t)a.n_pages};
    // a dimension of one element has no stride to speak of
    cuuint64_t strides[3] = {(cuuint64_t)a.token_b, (cuuint64_t)(a.Hk > 1 ? a.head_b : 16), (cuuint64_t)(a.n_pages > 1 ? a.page_b : 16)};
    for (const cuuint64_t s : strides)
        if (s == 0 || s >= (1ull << 40)) return false;
    cuuint32_t box[4] = {F8 ? D : 64, (cuuint32_t)std::min(ps, AC_TK), 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return encoder()(m, F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint8_t*>(base), dims,
                     strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, F8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_attn_join(const AttnArgs& a, int sms, int n_hdr, int rows, float lift, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    const bool list = rows > 16;
    cfg.gridDim = list ? dim3(4 * sms) : dim3(n_hdr, 8);
    cfg.blockDim = dim3(32 * ATT_JOIN_WARPS);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // it starts early and waits on the device
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return list ? cudaLaunchKernelEx(&cfg, k_attn_join<D, true>, a, n_hdr, rows, lift)
                : cudaLaunchKernelEx(&cfg, k_attn_join<D, false>, a, n_hdr, rows, lift);
}

template <int D, bool F8, int NTW, int RW, int KW>
cudaError_t launch_attn_rows(const AttnArgs& a, int sms, cudaStream_t st) {
    using C = AttCfg<D, F8, NTW, RW, KW>;
    static_assert(C::PER_SM * C::ROWS <= ATT_PART_ROWS && C::PER_SM <= ATT_MAX_PER_SM, "the workspace holds every CTA's partial sums");
    const int grid = std::min(sms, ATT_MAX_SMS) * C::PER_SM;
    k_attn_rows<D, F8, NTW, RW, KW><<<grid, C::NTH, C::SMEM, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? launch_attn_join<D>(a, sms, grid, C::ROWS, F8 ? 10.f : 0.f, st) : e;
}

template <int D, bool F8>
cudaError_t launch_attn_chunk(AttnArgs a, int sms, cudaStream_t st) {
    static_assert(AC_ROWS <= ATT_PART_ROWS, "the workspace holds every CTA's partial sums");
    const int grid = std::min(sms, ATT_MAX_SMS);
    CUtensorMap tk{}, tv{};
    a.tma = tmap_cache<D, F8>(&tk, a.k, a) && tmap_cache<D, F8>(&tv, a.v, a);
    constexpr int S = AcCfg<D, F8>::SMEM;
    switch ((a.softcap > 0.f ? 2 : 0) | (a.slopes ? 1 : 0)) {
        case 0: k_attn_chunk<D, F8, 0><<<grid, AC_THREADS, S, st>>>(tk, tv, a); break;
        case 1: k_attn_chunk<D, F8, 1><<<grid, AC_THREADS, S, st>>>(tk, tv, a); break;
        case 2: k_attn_chunk<D, F8, 2><<<grid, AC_THREADS, S, st>>>(tk, tv, a); break;
        default: k_attn_chunk<D, F8, 3><<<grid, AC_THREADS, S, st>>>(tk, tv, a);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? launch_attn_join<D>(a, sms, grid, AC_ROWS, F8 ? 6.f : 0.f, st) : e;
}
// Which kernel.  `rows`: the most rows of one request that share a cached head.  Up to 16 the row
// kernels read the cache at memory speed and waste no tensor work on absent rows (64 requests of 8 rows
// at 32K: 185 us, the chunk kernel 383; of 16 rows at 16K: 242 us, 278).  Above, the chunk kernel does
// (48 windows of 24 rows at 20K: 144 us, row kernel 196, capped at 30: 316 us, 445; 64 of 40 rows at 16K:
// 305 us, 520), except that it takes longer to start and end, so a small call (query rows x keys the table
// can hold below 2^19) stays with the row kernels (5 tokens of 8 heads a cached one at 1,000 keys: 15.4 us,
// the chunk kernel 22; 37 tokens at 8,192: 39 us, 34).  The bound is on what the table can hold because
// only the device knows the lengths.
template <int D, bool F8>
cudaError_t launch_attn(const AttnArgs& a, int sms, cudaStream_t st) {
    const int64_t rows = (int64_t)std::min(a.max_q, a.T) * a.G;
    if (rows <= 8) return launch_attn_rows<D, F8, 1, 1, 4>(a, sms, st);
    if (rows <= 16) return launch_attn_rows<D, F8, 2, 1, 4>(a, sms, st);
    const int64_t keys = std::min((int64_t)a.width * a.page_size, (int64_t)MOE_ATTN_MAX_KV);
    const bool small = (int64_t)a.T * a.G * keys < 1 << 19;
    if (rows <= 32 && small) return launch_attn_rows<D, F8, 2, 2, 2>(a, sms, st);
    return small ? launch_attn_rows<D, F8, 2, 4, 2>(a, sms, st) : launch_attn_chunk<D, F8>(a, sms, st);
}

int run_attn(const AttnCall& c) {
    int sms = 0;
    const int rc = attn_init(&sms);
    if (rc) return rc;
    const moe_kv_desc* d = c.d;
    const int64_t es = d->kv_type == MOE_KV_BF16 ? 2 : 1;
    const AttnWs L = attn_ws(d->head_dim);
    AttnArgs a{};
    a.q = c.q; a.q_stride = c.q_stride;
    a.k = static_cast<const uint8_t*>(d->k_cache); a.v = static_cast<const uint8_t*>(d->v_cache);
    a.k_scale = d->k_scale; a.v_scale = d->v_scale;
    a.page_b = d->page_stride * es; a.token_b = d->token_stride * es; a.head_b = d->head_stride * es;
    a.n_pages = d->n_pages; a.page_size = d->page_size;
    a.cu = c.cu; a.kv_len = c.kv_len; a.table = c.table; a.width = c.width;
    a.T = c.T; a.B = c.B; a.Hk = d->n_kv_heads; a.G = d->n_heads / d->n_kv_heads; a.max_q = c.max_q;
    // a window of all the keys there can be is none, and below it `position - window` stays within 32 bits
    // (positions are negative for rows before the first key)
    a.window = c.window >= MOE_ATTN_MAX_KV ? 0 : c.window;
    a.scale = c.scale; a.softcap = c.softcap; a.slopes = c.slopes; a.prefix = c.prefix;
    a.out = c.out; a.lse = c.lse;
    a.hdr = reinterpret_cast<int4*>(c.ws + L.hdr);
    a.ml = reinterpret_cast<float2*>(c.ws + L.ml);
    a.part = reinterpret_cast<float*>(c.ws + L.part);
    cudaError_t e;
    if (d->kv_type == MOE_KV_BF16)
        e = d->head_dim == 64 ? launch_attn<64, false>(a, sms, c.st) : launch_attn<128, false>(a, sms, c.st);
    else
        e = d->head_dim == 64 ? launch_attn<64, true>(a, sms, c.st) : launch_attn<128, true>(a, sms, c.st);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    count(2);
    return cuda_rc(cudaGetLastError());
}

}  // namespace

extern "C" {

int moe_kv_map(const int32_t* kv_len, const int32_t* q_len, int B, int page_size, const int32_t* free_pages, int n_free,
               int32_t* block_table, int table_width, int T, int32_t* kv_len_new, int32_t* cu_q, int32_t* position,
               int32_t* slot, int32_t* n_used, void* stream) {
    if (B < 0 || B > MOE_ATTN_MAX_B || T < 0 || T > MOE_KV_MAP_MAX_T || page_size < 1 || n_free < 0 || table_width < 1)
        return MOE_ERR_RANGE;
    if (B > 0 && (!kv_len || !q_len || !block_table || !kv_len_new)) return MOE_ERR_ARG;
    if (!cu_q || !n_used) return MOE_ERR_ARG;
    if ((!free_pages && n_free > 0) || ((!position || !slot) && T > 0)) return MOE_ERR_ARG;
    for (const void* p : {(const void*)kv_len, (const void*)q_len, (const void*)free_pages, (const void*)block_table,
                          (const void*)kv_len_new, (const void*)cu_q, (const void*)position, (const void*)slot,
                          (const void*)n_used})
        if (!aligned(p, 4)) return MOE_ERR_ARG;
    // every CTA reads the inputs while others write the outputs: none may share memory
    const void* const in[3] = {kv_len, q_len, free_pages};
    const size_t in_n[3] = {(size_t)B * 4, (size_t)B * 4, (size_t)n_free * 4};
    const void* const outp[6] = {block_table, kv_len_new, cu_q, position, slot, n_used};
    const size_t out_n[6] = {(size_t)B * table_width * 4, (size_t)B * 4, (size_t)(B + 1) * 4, (size_t)T * 4, (size_t)T * 4, 4};
    for (int o = 0; o < 6; ++o) {
        for (int i = 0; i < 3; ++i)
            if (overlap(outp[o], out_n[o], in[i], in_n[i])) return MOE_ERR_ARG;
        for (int i = 0; i < o; ++i)
            if (overlap(outp[o], out_n[o], outp[i], out_n[i])) return MOE_ERR_ARG;
    }
    KvMapArgs a{kv_len, q_len, free_pages, B, page_size, n_free, table_width, T,
                block_table, kv_len_new, cu_q, position, slot, n_used};
    const int grid = std::min(std::max(1, (T + KM_THREADS - 1) / KM_THREADS), 2 * 148);
    k_kv_map<<<grid, KM_THREADS, (size_t)2 * (B + 1) * 4, static_cast<cudaStream_t>(stream)>>>(a);
    count(1);
    return cuda_rc(cudaGetLastError());
}

int moe_rope_inv_freq(int kind, int rot_dim, double base, double factor, double original_len, double beta_fast,
                      double beta_slow, float* inv_freq, float* rot_scale) {
    if (!inv_freq || !rot_scale) return MOE_ERR_ARG;
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > 65536) return MOE_ERR_SHAPE;
    if (!(base > 1.0) || !isfinite(base) || kind < MOE_ROPE_PLAIN || kind > MOE_ROPE_PARTS) return MOE_ERR_RANGE;
    if (kind != MOE_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return MOE_ERR_RANGE;
    if (kind == MOE_ROPE_BASE && rot_dim < 4) return MOE_ERR_SHAPE;
    if (kind == MOE_ROPE_PARTS &&
        (!(original_len > 0.0) || !isfinite(original_len) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast)))
        return MOE_ERR_RANGE;
    if (kind == MOE_ROPE_BASE) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (kind == MOE_ROPE_LINEAR) f /= factor;
        if (kind == MOE_ROPE_PARTS) {
            const double turns = original_len * f / 6.283185307179586;
            const double keep = std::min(1.0, std::max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
            f = f * keep + f / factor * (1.0 - keep);
        }
        inv_freq[i] = (float)f;
    }
    *rot_scale = kind == MOE_ROPE_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return MOE_OK;
}

int moe_qk_norm_rope(const moe_kv_desc* kv, const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                     const uint16_t* v, int64_t v_stride, int T, const int32_t* position, const int32_t* slot,
                     const float* q_norm, const float* k_norm, float eps, const float* inv_freq, int rot_dim,
                     int interleaved, float rot_scale, uint16_t* q_out, int64_t out_stride, void* stream) {
    int rc = check_kv_desc(kv);
    if (rc) return rc;
    if (T < 0 || T > MOE_KV_MAP_MAX_T || !(eps >= 0.f) || !isfinite(eps) || !isfinite(rot_scale)) return MOE_ERR_RANGE;
    const int D = kv->head_dim;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16) return MOE_ERR_SHAPE;
    const int64_t qw = (int64_t)kv->n_heads * D, kw = (int64_t)kv->n_kv_heads * D;
    if (q_stride < qw || out_stride < qw || k_stride < kw || v_stride < kw) return MOE_ERR_SHAPE;
    if (q_stride % 8 || out_stride % 8 || k_stride % 8 || v_stride % 8) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;  // the buffers may be null
    if (!q || !k || !v || !position || !slot || !q_out || (rot_dim > 0 && !inv_freq)) return MOE_ERR_ARG;
    for (const void* p : {(const void*)q, (const void*)k, (const void*)v, (const void*)q_out})
        if (!aligned(p, 16)) return MOE_ERR_ARG;
    for (const void* p : {(const void*)position, (const void*)slot, (const void*)inv_freq})
        if (!aligned(p, 4)) return MOE_ERR_ARG;
    if (!aligned(q_norm, 16) || !aligned(k_norm, 16)) return MOE_ERR_ARG;
    // in place (the same rows) is fine: a thread reads its piece of a head before it writes it.  Rows that merely
    // overlap are not, nor queries written over keys or values, which other warps still read
    if ((q_out != q || out_stride != q_stride) && rows_overlap(q, q_stride, qw, q_out, out_stride, qw, T)) return MOE_ERR_ARG;
    if (rows_overlap(k, k_stride, kw, q_out, out_stride, qw, T) || rows_overlap(v, v_stride, kw, q_out, out_stride, qw, T))
        return MOE_ERR_ARG;
    RopeArgs a{};
    a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.out_stride = out_stride;
    a.q_out = q_out; a.position = position; a.slot = slot;
    a.q_norm = q_norm; a.k_norm = k_norm; a.inv_freq = inv_freq; a.k_scale = kv->k_scale; a.v_scale = kv->v_scale;
    a.eps = eps; a.rot_scale = rot_scale; a.T = T; a.Hq = kv->n_heads; a.Hk = kv->n_kv_heads; a.rot = rot_dim;
    a.interleaved = interleaved != 0;
    const int64_t es = kv->kv_type == MOE_KV_BF16 ? 2 : 1;
    a.k_cache = static_cast<uint8_t*>(kv->k_cache); a.v_cache = static_cast<uint8_t*>(kv->v_cache);
    a.page_b = kv->page_stride * es; a.token_b = kv->token_stride * es; a.head_b = kv->head_stride * es;
    a.page_size = kv->page_size; a.n_slots = (int64_t)kv->n_pages * kv->page_size;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f8 = kv->kv_type == MOE_KV_E4M3;
    if (D == 64) f8 ? launch_rope<64, true>(a, st) : launch_rope<64, false>(a, st);
    else f8 ? launch_rope<128, true>(a, st) : launch_rope<128, false>(a, st);
    count(1);
    return cuda_rc(cudaGetLastError());
}

size_t moe_attn_workspace_bytes(int T, int B, int n_heads, int n_kv_heads, int head_dim) {
    if (T < 0 || T > MOE_ATTN_MAX_B * MOE_DECODE_MAX_T || B < 0 || B > MOE_ATTN_MAX_B) return 0;
    if (n_heads < 1 || n_heads > MOE_ATTN_MAX_HEADS || n_kv_heads < 1 || n_heads % n_kv_heads) return 0;
    if (head_dim != 64 && head_dim != 128) return 0;
    return attn_ws(head_dim).total;
}

int moe_attn_decode(const moe_kv_desc* kv, const uint16_t* q, int64_t q_stride, int T, const int32_t* cu_q,
                    const int32_t* kv_len, int B, const int32_t* block_table, int table_width, int max_q, float scale,
                    float softcap, int window, const float* slopes, const int32_t* prefix, uint16_t* out, float* lse,
                    void* ws, size_t ws_bytes, void* stream) {
    if (max_q > MOE_DECODE_MAX_T) return MOE_ERR_RANGE;
    const AttnCall c{kv, q, q_stride, T, B, cu_q, kv_len, block_table, table_width, max_q, scale, softcap, window, slopes,
                     prefix, out, lse, static_cast<uint8_t*>(ws), ws_bytes, static_cast<cudaStream_t>(stream)};
    const int rc = check_attn(c, MOE_ATTN_MAX_B * MOE_DECODE_MAX_T);
    if (rc) return rc;
    return T == 0 || B == 0 ? MOE_OK : run_attn(c);
}

int moe_attn_prefill(const moe_kv_desc* kv, const uint16_t* q, int64_t q_stride, int T, const int32_t* cu_q,
                     const int32_t* kv_len, int B, const int32_t* block_table, int table_width, float scale,
                     float softcap, int window, const float* slopes, const int32_t* prefix, uint16_t* out, float* lse,
                     void* ws, size_t ws_bytes, void* stream) {
    const AttnCall c{kv, q, q_stride, T, B, cu_q, kv_len, block_table, table_width, std::max(T, 1), scale, softcap, window,
                     slopes, prefix, out, lse, static_cast<uint8_t*>(ws), ws_bytes, static_cast<cudaStream_t>(stream)};
    const int rc = check_attn(c, MOE_PREFILL_MAX_T);
    if (rc) return rc;
    return T == 0 || B == 0 ? MOE_OK : run_attn(c);
}

}  // extern "C"
