// Attention over the paged key-value cache.  For a query row (token i of
// request b, head) at position pos = kv_len - n_new + i (n_new: all its rows in the step), over its visible keys
// j in [lo, hi), hi = max(pos + 1, min(prefix, kv_len)), lo = max(0, pos - W + 1):
//   s_j = scale q . k_j, capped: cap tanh(s_j / cap), less slope |pos - j|
//   out = sum_j exp(s_j) v_j / sum_j exp(s_j),  lse = log sum_j exp(s_j).
// One pass over the keys with a running maximum and sum, all of it fp32.
//
// The rows of a request that share a cached head (its new tokens x the group of
// G = heads / kv_heads query heads, row = token * G + g) are cut into row tiles;
// a row tile and a cached head is an item, and an item is a run of key tiles.
// All key tiles of the call, in order, are dealt out evenly: each CTA of a grid
// that fills the GPU takes the same number of consecutive tiles, whatever the
// lengths, which only the device knows.  An item that falls into one CTA is
// written by it; one that is cut leaves fp32 partial sums, which a second kernel
// joins in order (so results do not depend on timing).
#pragma once

#include <type_traits>

#include "common.cuh"

#define ATT_MAX_SMS 152         // the workspace is sized for a grid of this many SMs
#define ATT_MAX_PER_SM 3        // and so many CTAs on each
#define ATT_PART_ROWS 256       // rows of partial sums per SM and slot
#define ATT_JOIN_WARPS 8

struct AttnArgs {
    const uint16_t* q;
    int64_t q_stride;  // elements from token to token
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    int64_t page_b, token_b, head_b;  // bytes
    int n_pages, page_size;
    const int32_t *cu, *kv_len, *table;
    int width, T, B, Hk, G, max_q, window, tma;
    float scale, softcap;
    const float* slopes;
    const int32_t* prefix;
    uint16_t* out;
    float* lse;
    float* part;   // [2 * CTAs][rows][D]
    float2* ml;    // [2 * CTAs][rows]: exponent reference (base 2) and sum
    int4* hdr;     // [CTAs]: {parts | rows << 16, first token, row of the request, cached head} of the item cut at this CTA's end
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)));
    return r;
}

// The cap of a base-2 score x, cap tanh(x / cap).  For y = x / cap up to 0.35 it is x + x z q(z), z = y^2, q a least-
// squares fit of tanh at Chebyshev nodes, within 9.9e-8 of y in fp32: the error is the score's own rounding whatever
// the cap (z = 0 leaves x as it is).  Above, cap (1 - 2 / (1 + e^2y)), whose error is 2^-23 of the cap, there of the
// score's size.  (For small y it would not be: 1e-7 of a cap of 1e6 is 0.1.)
struct AttCap {
    float in, out;  // ln 2 / cap (so that y = x in), cap log2 e
    __device__ __forceinline__ explicit AttCap(float cap) : in(0.6931471805599453f / cap), out(cap * 1.4426950408889634f) {}
    __device__ __forceinline__ float2 operator()(float2 x) const {
        const float2 y = fma2(x, both(in), both(0.f)), z = fma2(y, y, both(0.f));
        float2 q = fma2(z, both(-0.04913432523608208f), both(0.13299560546875f));
        q = fma2(q, z, both(-0.333326518535614f));
        q = fma2(fma2(x, z, both(0.f)), q, x);
        auto large = [&](float v) { return fmaf(-2.f * out, rcp_approx(1.f + ex2(v * (2.f * 1.4426950408889634f))), out); };
        return make_float2(fabsf(y.x) <= 0.35f ? q.x : large(y.x), fabsf(y.y) <= 0.35f ? q.y : large(y.y));
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 8 x 8 transpose of 16-bit elements across the warp
__device__ __forceinline__ uint32_t mat_t(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8); A and B fp16 or bf16
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// two e4m3 (low 16 bits) -> two fp16, exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
    uint32_t y;
    asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// A request's rows and lengths, with every device-side number clamped to what the call's arguments allow.
// Positions go by all the rows that the offsets give the request, also where only max_q of them are taken.
struct AttSeq {
    int t0, n, p0, pre;  // first row, rows, position of the first, end of the prefix
};
__device__ __forceinline__ AttSeq att_seq(const AttnArgs& a, int b) {
    AttSeq s;
    s.t0 = min(max(a.cu[b], 0), a.T);
    const int rows = min(max(a.cu[b + 1], s.t0), a.T) - s.t0;
    const int kv = min(max(a.kv_len[b], 0), (int)min((int64_t)a.width * a.page_size, (int64_t)MOE_ATTN_MAX_KV));
    s.n = min(rows, a.max_q);
    s.p0 = kv - rows;
    s.pre = a.prefix ? min(max(a.prefix[b], 0), kv) : 0;
    return s;
}
// visible keys [lo, hi) of token i of the request
__device__ __forceinline__ void att_range(const AttnArgs& a, const AttSeq& s, int i, int& lo, int& hi) {
    const int pos = s.p0 + i;
    hi = max(max(pos + 1, s.pre), 0);
    lo = a.window ? max(0, pos - a.window + 1) : 0;
}

// An item's position in the deal: row tile rt of request b for cached head h, key tile `tile` of n.
struct AttCur {
    int b, rt, h, tile, n, lo, hi;  // lo: where the key tiles start
    int first;                      // the first key that a row sees (lo rounded up again)
    AttSeq s;
};

// Key tiles of a row tile; they start at the first visible key, or at the multiple of ALIGN at or before it.
template <int ROWS, int TK, int ALIGN>
__device__ __forceinline__ int att_tiles(const AttnArgs& a, const AttSeq& s, int rt, int& first, int& lo, int& hi) {
    const int i0 = rt * ROWS / a.G, i1 = min(s.n - 1, (rt * ROWS + ROWS - 1) / a.G);
    int l1, h0;
    att_range(a, s, i0, first, h0);
    att_range(a, s, i1, l1, hi);
    lo = first - first % ALIGN;
    return hi > lo ? (hi - lo + TK - 1) / TK : 1;  // a row tile without a key still has its rows to write
}

template <int ROWS, int TK, int ALIGN>
__device__ __forceinline__ void att_enter(const AttnArgs& a, AttCur& c) {
    c.n = att_tiles<ROWS, TK, ALIGN>(a, c.s, c.rt, c.first, c.lo, c.hi);
}

// Next item in the deal's order (cached heads of a row tile, row tiles, requests), and next key tile.
template <int ROWS, int TK, int ALIGN>
__device__ __forceinline__ void att_next_item(const AttnArgs& a, AttCur& c) {
    c.tile = 0;
    if (++c.h < a.Hk) return;
    c.h = 0;
    if ((++c.rt) * ROWS >= c.s.n * a.G) {
        c.rt = 0;
        do {
            if (++c.b >= a.B) return;
            c.s = att_seq(a, c.b);
        } while (c.s.n == 0);
    }
    att_enter<ROWS, TK, ALIGN>(a, c);
}

template <int ROWS, int TK, int ALIGN>
__device__ __forceinline__ void att_next(const AttnArgs& a, AttCur& c) {
    if (++c.tile == c.n) att_next_item<ROWS, TK, ALIGN>(a, c);
}

// The deal: total, share per CTA, and where this CTA starts, in tiles, an item counting OV
// tiles more than it has (what beginning and ending it costs).  Every CTA computes it for
// itself: one read of the lengths into shared memory, then two block scans, row tiles per
// request and key tiles per row tile.  `scratch`: att_deal_bytes(B) of shared memory.
#define ATT_DEAL_SEQS 1024  // requests whose lengths are kept there; more are read again
constexpr __host__ __device__ int att_deal_bytes(int B) {
    return 16 * (B < ATT_DEAL_SEQS ? B : ATT_DEAL_SEQS) + 8 * 32 + 4 * (B + 1);
}

template <int ROWS, int TK, int NTH, int ALIGN, int OV>
__device__ __forceinline__ void att_deal(const AttnArgs& a, uint8_t* scratch, AttCur& c, int64_t& w0, int64_t& per, int64_t& total,
                                         int64_t& start) {
    if (a.B == 1 && (int64_t)min(a.T, a.max_q) * a.G <= ROWS) {  // one row tile at most: nothing to scan
        c.b = c.rt = 0;
        c.s = att_seq(a, 0);
        total = 0;
        per = 1;
        w0 = blockIdx.x;
        if (c.s.n == 0) return;
        att_enter<ROWS, TK, ALIGN>(a, c);
        total = (int64_t)(c.n + OV) * a.Hk;
        per = (total + gridDim.x - 1) / gridDim.x;
        w0 = per * blockIdx.x;
        c.h = (int)(w0 / (c.n + OV));
        start = (int64_t)c.h * (c.n + OV);
        c.tile = (int)max(w0 - start - OV, (int64_t)0);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int4* const seq = reinterpret_cast<int4*>(scratch);
    const int kept = min(a.B, ATT_DEAL_SEQS);
    int64_t* const red = reinterpret_cast<int64_t*>(scratch + 16 * kept);
    int* const base = reinterpret_cast<int*>(scratch + 16 * kept + 8 * 32);  // first row tile of each request
    __shared__ int s_b, s_rt;
    __shared__ int64_t s_before;
    auto get = [&](int b) {
        if (b >= kept) return att_seq(a, b);
        const int4 v = seq[b];
        return AttSeq{v.x, v.y, v.z, v.w};
    };
    auto scan = [&](int64_t v, int64_t& all) {  // exclusive over the block
        int64_t inc = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t t = __shfl_up_sync(~0u, inc, d);
            if (lane >= d) inc += t;
        }
        __syncthreads();
        if (lane == 31) red[warp] = inc;
        __syncthreads();
        int64_t ex = inc - v;
        all = 0;
#pragma unroll 4
        for (int w = 0; w < NTH / 32; ++w) {
            const int64_t t = red[w];
            if (w < warp) ex += t;
            all += t;
        }
        return ex;
    };
    const int ipt = (a.B + NTH - 1) / NTH, b0 = min(a.B, tid * ipt), b1 = min(a.B, b0 + ipt);
    int64_t mine = 0, entries;
    for (int b = b0; b < b1; ++b) {
        const AttSeq s = att_seq(a, b);
        if (b < kept) seq[b] = make_int4(s.t0, s.n, s.p0, s.pre);
        mine += ((int64_t)s.n * a.G + ROWS - 1) / ROWS;
    }
    int64_t ex = scan(mine, entries);
    for (int b = b0; b < b1; ++b) {
        base[b] = (int)ex;
        ex += ((int64_t)get(b).n * a.G + ROWS - 1) / ROWS;
    }
    if (tid == 0) base[a.B] = (int)entries;
    __syncthreads();
    const int ept = (int)((entries + NTH - 1) / NTH), e0 = min((int)entries, tid * ept), e1 = min((int)entries, e0 + ept);
    int first_b = 0;  // the last request that starts at or before entry e0
    if (e0 < e1)
        for (int lo = 0, hi = a.B; hi - lo > 1;) {
            const int mid = (lo + hi) >> 1;
            if (base[mid] <= e0) lo = mid;
            else hi = mid;
            first_b = lo;
        }
    // calls f(request, row tile, units) for this thread's entries until it returns true
    auto each = [&](auto f) {
        int b = first_b;
        AttSeq s = get(b);
        for (int e = e0; e < e1; ++e) {
            if (e >= base[b + 1]) {
                do ++b; while (base[b + 1] <= e);
                s = get(b);
            }
            int first, lo, hi;
            if (f(b, e - base[b], att_tiles<ROWS, TK, ALIGN>(a, s, e - base[b], first, lo, hi) + OV)) break;
        }
    };
    int64_t tiles = 0, all;
    each([&](int, int, int n) { tiles += n; return false; });
    const int64_t before = scan(tiles, all);
    total = all * a.Hk;
    per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)1);
    w0 = per * blockIdx.x;
    if (w0 < total) {
        const int64_t at = w0 / a.Hk;  // the entry that holds tile `at` of one head holds w0
        if (at >= before && at < before + tiles) {
            int64_t p = before;
            each([&](int b, int rt, int n) {
                if (at >= p + n) {
                    p += n;
                    return false;
                }
                s_b = b;
                s_rt = rt;
                s_before = p;
                return true;
            });
        }
        __syncthreads();
        c.b = s_b;
        c.rt = s_rt;
        c.s = get(c.b);
        att_enter<ROWS, TK, ALIGN>(a, c);
        const int64_t rem = w0 - s_before * a.Hk;
        c.h = (int)(rem / (c.n + OV));
        start = s_before * a.Hk + (int64_t)c.h * (c.n + OV);
        c.tile = (int)max(w0 - start - OV, (int64_t)0);
    }
}

template <int D, bool F8, int NTW, int RW, int KW>
struct AttCfg {
    static constexpr int ES = F8 ? 1 : 2, CH = D * ES / 16;     // 16-byte chunks of a cached row
    static constexpr int NTH = 32 * RW * KW, ROWS = 8 * NTW * RW;
    static constexpr int PER_SM = NTH > 128 ? 1 : NTW == 1 && !(F8 && D == 128) ? 3 : 2;
    static constexpr int WANT = RW == 2 ? 16384 : 32768;         // bytes of a stage
    static constexpr int TK = WANT / (2 * D * ES) > 128 ? 128 : WANT / (2 * D * ES);
    static constexpr int STAGE = 2 * TK * D * ES;
    static constexpr int ST = (PER_SM == 3 ? 65536 : RW == 2 ? 81920 : PER_SM == 2 ? 98304 : 163840) / STAGE;  // 2 to 10 stages
    static constexpr int KPW = TK / KW;                          // keys of a warp in a tile
    static constexpr int CK = F8 || KPW < 32 ? 16 : 32;           // and in one softmax step (e4m3: 32 spills)
    static constexpr int AROW = D + 4;                           // merge areas, one per row group, padded against bank conflicts
    static constexpr int AREA_B = 8 * NTW * AROW * 4;
    static constexpr int OFF_AREA = ST * STAGE, OFF_ML = OFF_AREA + RW * AREA_B;
    static constexpr int OFF_ROW = OFF_ML + RW * 8 * NTW * 8, SMEM = OFF_ROW + ST * TK * 8;
    static_assert(TK <= NTH || TK == 128, "one thread looks up one key");
    static_assert(PER_SM * (SMEM + 128 + 1024) <= 233472, "the CTAs of an SM share its 228 KB");
    static_assert(att_deal_bytes(MOE_ATTN_MAX_B) <= OFF_AREA, "the deal borrows the stages");
};

// One warp's share: RW row groups of 8 NTW rows x KW key groups.  The products
// are taken transposed, S^T = K Q^T and O^T += V^T P^T, so that the rows are the
// 8-wide side of mma.m16n8k16: a single query head wastes no more than 7 of 8
// columns, and K (as stored) and V (through ldmatrix.trans) are the A operands.
// e4m3 rows are widened to fp16, exactly; queries are then scaled by a power of
// two per row so that no bf16 value leaves fp16's range, and the softmax
// numerators by 2^10, so that those down to 2^-34 of the largest still count.
template <int D, bool F8, int NTW, int RW, int KW>
__global__ void __launch_bounds__(AttCfg<D, F8, NTW, RW, KW>::NTH, AttCfg<D, F8, NTW, RW, KW>::PER_SM)
    k_attn_rows(const AttnArgs a) {
    using C = AttCfg<D, F8, NTW, RW, KW>;
    constexpr int TK = C::TK, CH = C::CH, ES = C::ES, NTH = C::NTH, ROWS = C::ROWS, ST = C::ST, CK = C::CK;
    constexpr int SUB = CK / 16, MT = D / 16;
    constexpr float LOG2E = 1.4426950408889634f;
    constexpr float LIFT = F8 ? 10.f : 0.f;
    extern __shared__ __align__(128) uint8_t smem[];
    int64_t* offs = reinterpret_cast<int64_t*>(smem + C::OFF_ROW);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rw = warp % RW, kw = warp / RW, qd = lane & 3, g8 = lane >> 2;
    const uint32_t sb = smem_u32(smem);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    AttCur pre;
    int64_t w0, per, total, start;
    att_deal<ROWS, TK, NTH, 1, 0>(a, smem, pre, w0, per, total, start);
    const int my = (int)max((int64_t)0, min(per, total - w0));
    if (my == 0) {
        if (tid == 0) a.hdr[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    __syncthreads();  // the scan's shared memory is free
    AttCur cur = pre;

    // ---- loads: the page of tile p + 1 is fetched while tile p's row offsets are handed over
    int pg = 0, pg_off = 0, pg_head = 0;
    bool pg_live = false;
    int pre_n = 0;  // tiles whose page has been asked for
    auto fetch = [&] {
        if (pre_n < my && tid < TK) {
            const int key = pre.lo + pre.tile * TK + tid;
            pg_live = key < pre.hi;
            pg_head = pre.h;
            if (pg_live) {
                const int col = key / a.page_size;
                pg_off = key - col * a.page_size;
                pg = __ldg(a.table + (int64_t)pre.b * a.width + col);
            }
        }
        if (pre_n < my) {
            ++pre_n;
            if (pre_n < my) att_next<ROWS, TK, 1>(a, pre);
        }
    };
    auto hand_over = [&](int p) {
        if (p < my && tid < TK) {
            int64_t o = -1;
            if (pg_live) {
                if (pg >= 0 && pg < a.n_pages) o = pg * a.page_b + pg_off * a.token_b + pg_head * a.head_b;
                else moe_set_status(MOE_ERR_SLOT);  // its keys read as zeros
            }
            offs[(p % ST) * TK + tid] = o;
        }
    };
    auto issue = [&](int p) {
        if (p < my) {
            const uint32_t st = sb + (p % ST) * C::STAGE;
            const int c = tid % CH;
#pragma unroll
            for (int r0 = 0; r0 < TK; r0 += NTH / CH) {
                const int r = r0 + tid / CH;
                const int64_t o = offs[(p % ST) * TK + r];
                const int sw = CH >= 8 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3));
                const uint32_t dst = st + r * (CH * 16) + sw * 16;
                const int64_t src = (o < 0 ? 0 : o) + c * 16;
                cp_async16(dst, a.k + src, o >= 0);
                cp_async16(dst + TK * CH * 16, a.v + src, o >= 0);
            }
        }
        cp_async_commit();
    };
    fetch();
    for (int p = 0; p < ST - 1; ++p) {
        if (p < my) {
            hand_over(p);
            fetch();
            __syncthreads();
        }
        issue(p);
    }
    hand_over(ST - 1);
    fetch();

    // ---- state of an item
    uint32_t qf[NTW][MT][2];
    float acc[NTW][MT][4], m[NTW][2], l[NTW][2], rs[NTW][2], slope[NTW][2];
    int rlo[NTW][2], rhi[NTW][2], rpos[NTW][2];
    int all_lo = 0, all_hi = 0;  // keys that every row of the tile sees
    const bool extra = a.softcap > 0.f || a.slopes;
    const AttCap cap(a.softcap);
    float vs = 1.f;
    bool started = false;

    for (int it = 0; it < my; ++it) {
        cp_async_wait<ST - 2>();
        __syncthreads();
        issue(it + ST - 1);
        hand_over(it + ST);
        fetch();

        if (!started) {
            started = true;
            const float ks = (F8 && a.k_scale) ? __ldg(a.k_scale + cur.h) : 1.f;
            vs = (F8 && a.v_scale) ? __ldg(a.v_scale + cur.h) : 1.f;
            const int rows = min(ROWS, cur.s.n * a.G - cur.rt * ROWS);
            int t_lo, t_hi;
            att_range(a, cur.s, cur.rt * ROWS / a.G, t_lo, all_hi);
            att_range(a, cur.s, (cur.rt * ROWS + rows - 1) / a.G, all_lo, t_hi);
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt) {
                const int r = (rw * NTW + nt) * 8 + g8, rr = cur.rt * ROWS + r;
                const int i = rr / a.G, head = cur.h * a.G + rr % a.G;
                const uint16_t* qp = a.q + (int64_t)(cur.s.t0 + i) * a.q_stride + head * D;
                const bool live = r < rows;
#pragma unroll
                for (int k = 0; k < MT; ++k) {
                    if constexpr (F8) {
                        uint2 w = live ? *reinterpret_cast<const uint2*>(qp + k * 16 + qd * 4) : make_uint2(0, 0);
                        qf[nt][k][0] = w.x;
                        qf[nt][k][1] = w.y;
                    } else {
                        qf[nt][k][0] = live ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + qd * 2) : 0u;
                        qf[nt][k][1] = live ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + qd * 2 + 8) : 0u;
                    }
                }
                float unit = 1.f;
                if constexpr (F8) {  // bring the row's largest element to [2^14, 2^15)
                    float top = 0.f;
#pragma unroll
                    for (int k = 0; k < MT; ++k)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[nt][k][j] << 16)),
                                                   fabsf(__uint_as_float(qf[nt][k][j] & 0xffff0000u))));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    const int be = (int)(__float_as_uint(top) >> 23);
                    const int e = be == 255 ? 0 : max(be - 127 - 14, -100);
                    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                    unit = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                    for (int k = 0; k < MT; ++k)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            qf[nt][k][j] = pack_f16x2(__uint_as_float(qf[nt][k][j] << 16) * down,
                                                      __uint_as_float(qf[nt][k][j] & 0xffff0000u) * down);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {  // the rows of this lane's accumulators
                    const int r2 = (rw * NTW + nt) * 8 + qd * 2 + j, rr2 = cur.rt * ROWS + r2;
                    rs[nt][j] = a.scale * ks * __shfl_sync(~0u, unit, (qd * 2 + j) * 4) * LOG2E;
                    rlo[nt][j] = rhi[nt][j] = 0;
                    rpos[nt][j] = cur.s.p0 + rr2 / a.G;
                    slope[nt][j] = 0.f;
                    if (r2 < rows) {
                        att_range(a, cur.s, rr2 / a.G, rlo[nt][j], rhi[nt][j]);
                        if (a.slopes) slope[nt][j] = __ldg(a.slopes + cur.h * a.G + rr2 % a.G) * LOG2E;
                    }
                    m[nt][j] = -INFINITY;
                    l[nt][j] = 0.f;
                }
#pragma unroll
                for (int k = 0; k < MT; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[nt][k][j] = 0.f;
            }
        }

        // ---- one key tile
        const uint32_t st = sb + (it % ST) * C::STAGE, stv = st + TK * CH * 16;
        const int k0 = cur.lo + cur.tile * TK;
        const bool masked = k0 < all_lo || k0 + TK > all_hi;
        auto chunk_addr = [&](uint32_t base, int row, int c) {
            const int sw = CH >= 8 ? (c ^ (row & 7)) : (c ^ ((row >> 1) & 3));
            return base + row * (CH * 16) + sw * 16;
        };
#pragma unroll 1
        for (int kc = 0; kc < C::KPW; kc += CK) {
            const int kr = kw * C::KPW + kc;  // first key row of this step in the tile
            float s[NTW][SUB][4];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
#pragma unroll
                for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[nt][u][j] = 0.f;
                const int row = kr + u * 16 + (lane & 15);
                if constexpr (F8) {
#pragma unroll
                    for (int k2 = 0; k2 < MT / 2; ++k2) {
                        uint32_t r[4];
                        ldsm4(r, chunk_addr(st, row, k2 * 2 + (lane >> 4)));
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t fa[4] = {e4m3x2_to_f16x2(r[2 * h]), e4m3x2_to_f16x2(r[2 * h + 1]),
                                                    e4m3x2_to_f16x2(r[2 * h] >> 16), e4m3x2_to_f16x2(r[2 * h + 1] >> 16)};
#pragma unroll
                            for (int nt = 0; nt < NTW; ++nt)
                                mma16816<true>(s[nt][u], fa, qf[nt][2 * k2 + h][0], qf[nt][2 * k2 + h][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < MT; ++k) {
                        uint32_t fa[4];
                        ldsm4(fa, chunk_addr(st, row, k * 2 + (lane >> 4)));
#pragma unroll
                        for (int nt = 0; nt < NTW; ++nt) mma16816<false>(s[nt][u], fa, qf[nt][k][0], qf[nt][k][1]);
                    }
                }
            }
            // scores in base 2; this lane holds keys kr + 16 u + g8 (+ 8) of rows 2 qd and 2 qd + 1
            uint32_t pb[NTW][SUB][2];
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt) {
                if (extra) {
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            float2 x = make_float2(s[nt][u][e] * rs[nt][0], s[nt][u][e + 1] * rs[nt][1]);
                            if (a.softcap > 0.f) x = cap(x);
                            s[nt][u][e] = x.x;
                            s[nt][u][e + 1] = x.y;
                        }
                    if (a.slopes) {
#pragma unroll
                        for (int u = 0; u < SUB; ++u)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = e & 1, key = k0 + kr + u * 16 + g8 + (e >> 1) * 8;
                                s[nt][u][e] -= slope[nt][j] * fabsf((float)(rpos[nt][j] - key));
                            }
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[nt][u][e] *= rs[nt][e & 1];
                }
                if (masked) {
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = e & 1, key = k0 + kr + u * 16 + g8 + (e >> 1) * 8;
                            if (key < rlo[nt][j] || key >= rhi[nt][j]) s[nt][u][e] = -INFINITY;
                        }
                }
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top[e & 1] = fmaxf(top[e & 1], s[nt][u][e]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(~0u, top[j], d));
                }
                const bool grew = top[0] > m[nt][0] || top[1] > m[nt][1];
                if (__any_sync(~0u, grew)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float mn = fmaxf(m[nt][j], top[j]);
                        const float f = m[nt][j] == mn ? 1.f : ex2(m[nt][j] - mn);
                        m[nt][j] = mn;
                        l[nt][j] *= f;
#pragma unroll
                        for (int k = 0; k < MT; ++k) {
                            acc[nt][k][j] *= f;
                            acc[nt][k][2 + j] *= f;
                        }
                    }
                }
                const float ref[2] = {m[nt][0] == -INFINITY ? 0.f : m[nt][0] - LIFT, m[nt][1] == -INFINITY ? 0.f : m[nt][1] - LIFT};
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = ex2(s[nt][u][e] - ref[e & 1]);
                        l[nt][e & 1] += p[e];
                    }
                    // the numerators are rounded once more for the product with V, to bf16 (2^-8) or, beside e4m3
                    // values, fp16 (2^-11): an MMA takes one type, and fp32 values would need the tf32 form at half
                    // its rate and twice the registers; the sum above takes them unrounded
                    pb[nt][u][0] = mat_t(F8 ? pack_f16x2(p[0], p[1]) : pack_bf16x2(p[0], p[1]));
                    pb[nt][u][1] = mat_t(F8 ? pack_f16x2(p[2], p[3]) : pack_bf16x2(p[2], p[3]));
                }
            }
            // O^T += V^T P^T.  In a tile with masked places a zero numerator may meet an infinite or
            // NaN value that its row must not see: those values are taken out of the product here
            // and added below to the rows that do see them.
            bool odd = false;
            auto clean = [&](uint32_t x) {
                constexpr uint32_t EXP = F8 ? 0x7c00u : 0x7f80u;
                uint32_t keep = 0xffffffffu;
                if ((x & EXP) == EXP) keep &= 0xffff0000u;
                if (((x >> 16) & EXP) == EXP) keep &= 0x0000ffffu;
                odd |= keep != 0xffffffffu;
                return x & keep;
            };
            auto pv = [&](auto masked_tag) {
                constexpr bool MASKED = decltype(masked_tag)::value;
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    if constexpr (F8) {
#pragma unroll
                        for (int k2 = 0; k2 < MT / 2; ++k2) {
                            uint32_t r[4];
                            ldsm4t(r, chunk_addr(stv, kr + u * 16 + (lane & 15), k2 * 2 + (lane >> 4)));
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t x0 = e4m3x2_to_f16x2(r[2 * h]), x1 = e4m3x2_to_f16x2(r[2 * h] >> 16);
                                const uint32_t y0 = e4m3x2_to_f16x2(r[2 * h + 1]), y1 = e4m3x2_to_f16x2(r[2 * h + 1] >> 16);
                                uint32_t fa[4] = {__byte_perm(x0, x1, 0x5410), __byte_perm(x0, x1, 0x7632),
                                                  __byte_perm(y0, y1, 0x5410), __byte_perm(y0, y1, 0x7632)};
                                if constexpr (MASKED) {
#pragma unroll
                                    for (int e = 0; e < 4; ++e) fa[e] = clean(fa[e]);
                                }
#pragma unroll
                                for (int nt = 0; nt < NTW; ++nt)
                                    mma16816<true>(acc[nt][2 * k2 + h], fa, pb[nt][u][0], pb[nt][u][1]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < MT; ++k) {
                            uint32_t fa[4];
                            ldsm4t(fa, chunk_addr(stv, kr + u * 16 + (lane & 7) + (lane >> 4) * 8, k * 2 + ((lane >> 3) & 1)));
                            if constexpr (MASKED) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) fa[e] = clean(fa[e]);
                            }
#pragma unroll
                            for (int nt = 0; nt < NTW; ++nt) mma16816<false>(acc[nt][k], fa, pb[nt][u][0], pb[nt][u][1]);
                        }
                    }
                }
            };
            if (masked) pv(std::true_type{});
            else pv(std::false_type{});
            if (masked && __any_sync(~0u, odd)) {
#pragma unroll
                for (int k = 0; k < MT; ++k)
#pragma unroll
                    for (int d2 = 0; d2 < 2; ++d2) {
                        const int d = F8 ? k * 16 + g8 * 2 + d2 : k * 16 + g8 + d2 * 8;
#pragma unroll 1
                        for (int r = kr; r < kr + CK; ++r) {
                            const uint32_t at = chunk_addr(stv, r, d * ES / 16) - sb + (d * ES) % 16;
                            float x;
                            if constexpr (F8) {
                                const uint32_t hx = e4m3x2_to_f16x2(smem[at]);
                                x = half_bits_to_f32((uint16_t)hx);
                            } else {
                                x = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(smem + at));
                            }
                            if (fabsf(x) < INFINITY) continue;
#pragma unroll
                            for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    if (k0 + r >= rlo[nt][j] && k0 + r < rhi[nt][j]) acc[nt][k][2 * d2 + j] += x;
                        }
                    }
            }
        }

        // ---- the item ends here: join the key groups, write the rows or their partial sums
        const bool last = cur.tile == cur.n - 1;
        if (last || it == my - 1) {
            started = false;
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nt][j] += __shfl_xor_sync(~0u, l[nt][j], d);
                }
            float* const ar = reinterpret_cast<float*>(smem + C::OFF_AREA + rw * C::AREA_B);
            float2* const mls = reinterpret_cast<float2*>(smem + C::OFF_ML) + rw * 8 * NTW;
            auto dim = [&](int k, int d2) { return F8 ? k * 16 + g8 * 2 + d2 : k * 16 + g8 + d2 * 8; };
            auto put = [&] {
#pragma unroll
                for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = nt * 8 + qd * 2 + j;
                        if (g8 == 0) mls[r] = make_float2(m[nt][j], l[nt][j]);
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            ar[r * C::AROW + dim(t, 0)] = acc[nt][t][j];
                            ar[r * C::AROW + dim(t, 1)] = acc[nt][t][2 + j];
                        }
                    }
            };
#pragma unroll 1
            for (int from = 1; from < KW; ++from) {  // the first key group takes in the others, one at a time
                if (kw == from) put();
                __syncthreads();
                if (kw == 0) {
#pragma unroll
                    for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int r = nt * 8 + qd * 2 + j;
                            const float2 o = mls[r];
                            const float mn = fmaxf(m[nt][j], o.x);
                            const float f0 = m[nt][j] == mn ? 1.f : ex2(m[nt][j] - mn), f1 = o.x == mn ? 1.f : ex2(o.x - mn);
                            m[nt][j] = mn;
                            l[nt][j] = l[nt][j] * f0 + o.y * f1;
#pragma unroll
                            for (int t = 0; t < MT; ++t) {
                                acc[nt][t][j] = acc[nt][t][j] * f0 + ar[r * C::AROW + dim(t, 0)] * f1;
                                acc[nt][t][2 + j] = acc[nt][t][2 + j] * f0 + ar[r * C::AROW + dim(t, 1)] * f1;
                            }
                        }
                }
                if (from + 1 < KW) __syncthreads();
            }
            const int64_t at = w0 + it;
            const int64_t first = at - cur.tile;  // the item's first tile in the deal
            const bool whole = first >= w0 && last;
            const int rows = min(ROWS, cur.s.n * a.G - cur.rt * ROWS);
            if (kw == 0) {
                __syncwarp();
                put();
                __syncwarp();
                const int slot = 2 * blockIdx.x + (first >= w0 ? 1 : 0);
                for (int r = 0; r < 8 * NTW; ++r) {
                    const int rt = rw * 8 * NTW + r;
                    if (rt >= rows) break;
                    const float2 o = mls[r];
                    if (whole) {
                        const int rr = cur.rt * ROWS + rt;
                        const int64_t row = (int64_t)(cur.s.t0 + rr / a.G) * (a.Hk * a.G) + cur.h * a.G + rr % a.G;
                        const float f = o.y == 0.f ? 0.f : vs / o.y;
                        if (D == 128 || lane < 16) {
                            const float4 x = *reinterpret_cast<const float4*>(ar + r * C::AROW + lane * 4);
                            *reinterpret_cast<uint2*>(a.out + row * D + lane * 4) =
                                make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
                        }
                        if (a.lse && lane == 0)
                            a.lse[row] = o.y == 0.f ? -INFINITY : (o.x - LIFT + log2f(o.y)) * 0.6931471805599453f;
                    } else {
                        const int64_t row = (int64_t)slot * ROWS + rt;
                        if (D == 128 || lane < 16) {
                            float4 x = *reinterpret_cast<const float4*>(ar + r * C::AROW + lane * 4);
                            x.x *= vs; x.y *= vs; x.z *= vs; x.w *= vs;
                            *reinterpret_cast<float4*>(a.part + row * D + lane * 4) = x;
                        }
                        if (lane == 0) a.ml[row] = make_float2(o.x, o.y);
                    }
                }
            }
            if (it == my - 1 && tid == 0) {
                int parts = 0;
                if (!last && first >= w0) parts = (int)((first + cur.n - 1) / per - blockIdx.x) + 1;
                a.hdr[blockIdx.x] = make_int4(parts | rows << 16, cur.s.t0, cur.rt * ROWS, cur.h);
            }
        }
        if (it + 1 < my) att_next<ROWS, TK, 1>(a, cur);
    }
}

// Joins the parts of an item that starts in CTA c of the grid before and ends in a
// later one: part 0 in c's second slot, the others in the first slot of the CTAs
// after it, always in that order.  Units of work: four rows a warp for items of up
// to 8 parts (cut once or twice), a row a warp up to 32, a row a CTA above (a long
// cache and few rows).  LIST: every CTA numbers all units from the headers and one
// wave of CTAs does them; otherwise (few rows an item) CTA (c, y) takes every
// gridDim.y-th unit of item c, which saves the numbering (1 us of 12).  Bound by
// latency: the first parts of a row are asked for before their weights.
__device__ __forceinline__ int join_units(int x) {
    const int parts = x & 0xffff, rows = x >> 16;
    return parts == 0 ? 0 : parts <= 8 ? (rows + 4 * ATT_JOIN_WARPS - 1) / (4 * ATT_JOIN_WARPS)
                        : parts <= 32 ? (rows + ATT_JOIN_WARPS - 1) / ATT_JOIN_WARPS : rows;
}

template <int D, bool LIST>
__global__ void __launch_bounds__(32 * ATT_JOIN_WARPS, 4) k_attn_join(const AttnArgs a, int n_hdr, int rows_per, float lift) {
    constexpr int V = D / 32, AHEAD = 8, NTH = 32 * ATT_JOIN_WARPS;
    __shared__ float s_acc[ATT_JOIN_WARPS][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto unit_of = [&](const int c, const int4 h, const int nth_unit) {
        const int parts = h.x & 0xffff, rows = h.x >> 16;
        const bool few = parts <= 32;
        auto slot = [&](int p) { return (int64_t)(p == 0 ? 2 * c + 1 : 2 * (c + p)) * rows_per; };
        auto out_row = [&](int r) {
            const int rr = h.z + r;
            return (int64_t)(h.y + rr / a.G) * (a.Hk * a.G) + h.w * a.G + rr % a.G;
        };
        if (parts <= 8) {
            constexpr int L = D / 4, AT = 32 / L, N = 4 / AT;  // lanes a row, rows at a time, times
            const int q = lane >> 3, p8 = lane & 7;            // this lane's row and part of the 4 x 8 weights
            const int r0 = (nth_unit * ATT_JOIN_WARPS + warp) * 4;
            if (r0 < rows) {
                const bool live = p8 < parts && r0 + q < rows;
                const float2 o = live ? a.ml[slot(p8) + r0 + q] : make_float2(-INFINITY, 0.f);
                float4 x[N][2];
                auto load = [&](int n, int p) {
                    const int r = r0 + n * AT + lane / L;
                    return p < parts && r < rows ? *reinterpret_cast<const float4*>(a.part + (slot(p) + r) * D + (lane % L) * 4)
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
                };
    #pragma unroll
                for (int n = 0; n < N; ++n) {
                    x[n][0] = load(n, 0);
                    x[n][1] = load(n, 1);
                }
                float top = o.x;
    #pragma unroll
                for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                const float w = ex2(o.x - (top == -INFINITY ? 0.f : top));
                float sum = o.y * w;
    #pragma unroll
                for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                if (a.lse && p8 == 0 && r0 + q < rows)
                    a.lse[out_row(r0 + q)] = sum == 0.f ? -INFINITY : (top - lift + log2f(sum)) * 0.6931471805599453f;
    #pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int k = n * AT + lane / L, r = r0 + k;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int p = 0; p < parts; ++p) {
                        const float4 v = p < 2 ? (p ? x[n][1] : x[n][0]) : load(n, p);
                        const float f = __shfl_sync(~0u, w, k * 8 + p);
                        y.x += f * v.x; y.y += f * v.y; y.z += f * v.z; y.w += f * v.w;
                    }
                    const float f = __shfl_sync(~0u, inv, k * 8);
                    if (r < rows)
                        *reinterpret_cast<uint2*>(a.out + out_row(r) * D + (lane % L) * 4) =
                            make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
                }
            }
            return;
        }
        const int p0 = few ? 0 : warp, dp = few ? 1 : ATT_JOIN_WARPS;  // this warp's parts of a row
        const int r = few ? nth_unit * ATT_JOIN_WARPS + warp : nth_unit;
        if (r < rows) {  // (the same for the whole CTA where its warps meet below)
            float x[AHEAD][V];
            auto load = [&](int first) {
    #pragma unroll
                for (int n = 0; n < AHEAD; ++n) {
                    const int p = first + n * dp;
    #pragma unroll
                    for (int i = 0; i < V; ++i) x[n][i] = p < parts ? a.part[(slot(p) + r) * D + i * 32 + lane] : 0.f;
                }
            };
            load(p0);
            float top = -INFINITY;
            for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.ml[slot(p) + r].x);
    #pragma unroll
            for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            for (int p = lane; p < parts; p += 32) {
                const float2 o = a.ml[slot(p) + r];
                sum += o.y * ex2(o.x - ref);
            }
    #pragma unroll
            for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
            const int64_t row = out_row(r);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            float acc[V];
    #pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.f;
            for (int first = p0; first < parts; first += AHEAD * dp) {
                if (first > p0) load(first);
    #pragma unroll
                for (int n = 0; n < AHEAD; ++n) {
                    const int p = first + n * dp;
                    if (p >= parts) break;
                    const float f = ex2(a.ml[slot(p) + r].x - ref);
    #pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] += f * x[n][i];
                }
            }
            if (few) {
    #pragma unroll
                for (int i = 0; i < V; ++i) a.out[row * D + lane + i * 32] = f32_to_bf16_bits(acc[i] * inv);
            } else {
                __syncthreads();
    #pragma unroll
                for (int i = 0; i < V; ++i) s_acc[warp][lane + i * 32] = acc[i];
                __syncthreads();
                if (threadIdx.x < D) {
                    float y = 0.f;
    #pragma unroll
                    for (int w = 0; w < ATT_JOIN_WARPS; ++w) y += s_acc[w][threadIdx.x];
                    a.out[row * D + threadIdx.x] = f32_to_bf16_bits(y * inv);
                }
            }
            if (a.lse && (few ? lane : threadIdx.x) == 0)
                a.lse[row] = sum == 0.f ? -INFINITY : (top - lift + log2f(sum)) * 0.6931471805599453f;
        }
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (!LIST) {
        const int4 h = a.hdr[blockIdx.x];
        const int n = join_units(h.x);
        for (int u = blockIdx.y; u < n; u += gridDim.y) unit_of(blockIdx.x, h, u);
    } else {
        __shared__ int s_first[2 * NTH], s_sum[ATT_JOIN_WARPS];  // first unit of each header's item
        __shared__ int4 s_hdr[2 * NTH];
        static_assert(ATT_MAX_SMS * ATT_MAX_PER_SM <= 2 * NTH, "two headers a thread");
        int n2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int at = 2 * threadIdx.x + k;
            const int4 h = at < n_hdr ? a.hdr[at] : make_int4(0, 0, 0, 0);
            s_hdr[at] = h;
            n2[k] = join_units(h.x);
        }
        int inc = n2[0] + n2[1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(~0u, inc, d);
            if (lane >= d) inc += t;
        }
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        int before = inc - n2[0] - n2[1], units = 0;
#pragma unroll
        for (int w = 0; w < ATT_JOIN_WARPS; ++w) {
            if (w < warp) before += s_sum[w];
            units += s_sum[w];
        }
        s_first[2 * threadIdx.x] = before;
        s_first[2 * threadIdx.x + 1] = before + n2[0];
        __syncthreads();
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            int c = 0;
            for (int hi = 2 * NTH; hi - c > 1;) {  // the last header whose first unit is at or before this one
                const int mid = (c + hi) >> 1;
                if (s_first[mid] <= unit) c = mid;
                else hi = mid;
            }
            unit_of(c, s_hdr[c], unit - s_first[c]);
        }
    }
}
