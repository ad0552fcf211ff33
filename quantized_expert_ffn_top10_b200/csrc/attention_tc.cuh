// Attention on the 5th-generation tensor cores: row tiles of 2 x 128 rows
// (attention.cuh has the formulas, the items and the deal).
//
// Per key tile of 128 and half h of the rows: S_h = Q_h K^T (tcgen05.mma, both
// operands in shared memory, fp32 in TMEM), numerators P_h = exp2(S_h - m) by
// 128 threads, one row each, written over S_h in TMEM as 16-bit, and O_h += P_h V
// (A from TMEM, V as stored: keys x dims, an MN-major B operand).  The two halves
// alternate, so the tensor cores work on one while the other is in its softmax:
// QK0(j), PV1(j-1), QK1(j), PV0(j), ...  An item of at most 128 rows (a decode
// window, a short chunk) has both halves hold the same rows and take the key
// tiles in turn, QK0(j), PV1(j-1), QK1(j+1), PV0(j), ..., and adds them up at its
// end.  A commit covers everything issued before it, so S_h being ready also says
// that the half's last PV is done, and its threads may rescale O_h in place.  They
// do so only when a row's maximum has grown by more than 2^8 since its reference
// was taken: numerators stay below 2^8 (2^14 in fp16), which costs no precision,
// and after the first tiles it hardly ever happens.
//
// Roles (16 warps; warps 8 to 15 give registers up to the softmax): 0-3 and 4-7 the
// softmax of the two halves, 12 the MMAs, 13 the TMA loads (a box per page and 64
// columns), 8-11 what the loads need beside that: e4m3 rows widened to fp16 (exactly; the queries are then scaled per row by
// a power of two, as in the row kernel), non-finite values of partly masked V
// tiles set aside, and the whole gather, row by row, for page sizes that TMA boxes
// do not tile (not a power of two, or below 8).
#pragma once

#include <type_traits>

#include "attention.cuh"

#define AC_THREADS 512
#define AC_ROWS 256
#define AC_TK 128
// An item's beginning and end, in key tiles, for the deal.  A chunk's first rows are items of one tile or
// two, and the CTAs that get them end last unless this is counted: 8,192 tokens from the first, bf16 / e4m3:
// 495 / 692 us at 1, 412 / 582 at 2, 303 / 424 at 4, 292 / 342 at 6, 298 / 340 at 8, 303 / 346 at 10.
#define AC_OV 6

template <int D, bool F8>
struct AcCfg {
    static constexpr int TILE = AC_TK * D * 2;                // one 16-bit operand tile: a half of Q, K or V
    static constexpr int RAW = AC_TK * D;                     // one e4m3 tile as stored
    static constexpr int NS = D == 64 ? 8 : F8 ? 3 : 4;       // ring of operand tiles: K0 V0 K1 V1 ...
    static constexpr int NRAW = !F8 ? 0 : D == 64 ? 6 : 4;    // and of e4m3 tiles on their way into it
    static constexpr int OFF_RING = 2 * TILE, OFF_RAW = OFF_RING + NS * TILE;
    static constexpr int OFF_ROW = OFF_RAW;                   // gather: row offsets (no e4m3 tile is staged then)
    static constexpr int OFF_ML = OFF_RAW + (F8 ? NRAW * RAW : 2 * AC_TK * 8);
    static constexpr int OFF_BAR = OFF_ML + 128 * 8;
    static constexpr int SMEM = OFF_BAR + 448 + 1024;         // and room to align to 1024 bytes
    static_assert(SMEM <= 232448, "227 KB of shared memory per CTA");
};

// One lane of the warp, the same each time; true for it.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
    return ok != 0;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void reg_tie8(uint32_t* r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}
// no use of these registers is scheduled before this point (after a wait for the loads)
__device__ __forceinline__ void reg_tie32(uint32_t* r) {
#pragma unroll
    for (int i = 0; i < 32; i += 8) reg_tie8(r + i);
}

// 4D tiled bulk tensor load global -> shared; c0 is the innermost coordinate (elements).
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
            "r"(smem_u32(smem_dst)),
        "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// Shared-memory descriptor of V as stored, [dims / 64][128 keys][64 dims] with
// 128-byte rows, 128-byte swizzle, read with the dims as the operand's rows:
// 64-dim blocks AC_TK * 128 bytes apart (LBO), groups of 8 keys 1024 bytes (SBO).
__device__ __forceinline__ uint64_t make_sdesc_v(uint32_t smem_addr) {
    uint64_t d = make_sdesc_sw128(smem_addr);
    d &= ~((uint64_t)0x3FFF << 16);
    return d | (uint64_t)((AC_TK * 128) >> 4) << 16;
}

// kind::f16 instruction descriptor with fp32 accumulation; type 0 fp16, 1 bf16;
// b_mn: B is MN-major
constexpr __host__ __device__ uint32_t ac_idesc(int type, int N, bool b_mn) {
    return (1u << 4) | ((uint32_t)type << 7) | ((uint32_t)type << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((128u >> 4) << 24);
}

// tanh y / y - 1 = z q(z), z = y^2, for |y| <= 0.7: q a least-squares fit at Chebyshev nodes, within 4.6e-8 in fp32.
__device__ __forceinline__ float2 ac_cap_poly2(float2 z) {
    float2 q = fma2(z, both(0.0018368171295151114f), both(-0.007793231401592493f));
    q = fma2(q, z, both(0.02151893451809883f));
    q = fma2(q, z, both(-0.05390692502260208f));
    q = fma2(q, z, both(0.1333281248807907f));
    return fma2(q, z, both(-0.33333316445350647f));
}

// MODE: 1 slopes, 2 a cap, 3 both.  Each is kept out of the others' code, whose instructions would cost them 2 to 3%.
template <int D, bool F8, int MODE>
__global__ void __launch_bounds__(AC_THREADS, 1)
    k_attn_chunk(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const AttnArgs a) {
    using C = AcCfg<D, F8>;
    constexpr int TILE = C::TILE, NS = C::NS, NRAW = C::NRAW, BLK = AC_TK * 128;  // BLK: a 64-column block of a tile
    constexpr float LOG2E = 1.4426950408889634f, LIFT = F8 ? 6.f : 0.f, GROW = 8.f;
    constexpr uint32_t S_COL = 0, O_COL = 256;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    int64_t* const offs = reinterpret_cast<int64_t*>(smem + C::OFF_ROW);
    float2* const half_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    uint64_t* const bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t *const full = bar, *const empty = bar + NS, *const sfull = bar + 2 * NS, *const pfull = sfull + 2,
             *const qready = pfull + 2, *const ofull = qready + 1, *const half_up = ofull + 1, *const half_read = half_up + 1,
             *const rows_up = half_read + 1, *const cleaned = rows_up + 1, *const raw_full = cleaned + NS,
             *const raw_empty = raw_full + NRAW;
    uint32_t* const tm = reinterpret_cast<uint32_t*>(raw_empty + NRAW);
    volatile int* const odd = reinterpret_cast<int*>(tm + 2);  // [8]: 1 + the item whose masked tiles held non-finite values
    static_assert((3 * NS + 9 + 2 * NRAW) * 8 + 8 + 32 <= 448, "barriers");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, F8 || !a.tma ? 128 : 1);
            mbar_init(empty + i, 1);
            mbar_init(cleaned + i, 128);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(sfull + h, 1);
            mbar_init(pfull + h, 4);
        }
        mbar_init(qready, 8);
        mbar_init(ofull, 1);
        mbar_init(half_up, 4);
        mbar_init(half_read, 4);
        mbar_init(rows_up, 128);
        for (int i = 0; i < NRAW; ++i) {
            mbar_init(raw_full + i, 1);
            mbar_init(raw_empty + i, 128);
        }
        fence_mbar_init();
        for (int i = 0; i < 8; ++i) odd[i] = 0;
    }
    if (warp == 12) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    AttCur cur;
    int share, span, rel;  // the deal's tiles per CTA; this CTA's; where the item at `cur` starts, from this CTA's first
    {
        int64_t w0, per, total, start;
        static_assert(att_deal_bytes(MOE_ATTN_MAX_B) <= C::OFF_ML, "the deal borrows the tiles");
        att_deal<AC_ROWS, AC_TK, AC_THREADS, AC_TK, AC_OV>(a, smem, cur, w0, per, total, start);
        const bool fits = per < (1 << 30);  // or not in years
        share = fits ? (int)per : 1;
        span = fits ? (int)max(min(per, total - w0), (int64_t)0) : 0;
        rel = (int)(start - w0);
        if (tid == 0) {
            a.hdr[blockIdx.x] = make_int4(0, 0, 0, 0);
            if (!fits) moe_set_status(MOE_ERR_RANGE);
        }
    }
    tc_fence_before();
    __syncthreads();  // barriers and TMEM are there, and the deal's shared memory is free
    tc_fence_after();
    const uint32_t tmem = *tm;

    // This CTA's piece of an item: its key tiles [cur.tile, cur.tile + cnt).  next_piece() steps to the
    // item after `cur` unless it is the first call, and past items of which only the overhead is dealt here.
    int cnt = 0;
    auto next_piece = [&] {
        if (span == 0) return false;
        for (bool on = cnt == 0;; on = false) {
            if (!on) {
                rel += cur.n + AC_OV;
                if (rel >= span) return false;
                att_next_item<AC_ROWS, AC_TK, AC_TK>(a, cur);
            }
            cur.tile = max(-rel - AC_OV, 0);
            cnt = min(span - rel - AC_OV, cur.n) - cur.tile;
            if (cnt > 0) return true;
        }
    };
    auto rows_of = [&] { return min(AC_ROWS, cur.s.n * a.G - cur.rt * AC_ROWS); };
    // keys that every row of the item sees: [lo, hi); a tile not inside is masked somewhere
    auto seen_by_all = [&](int& lo, int& hi) {
        int x;
        att_range(a, cur.s, cur.rt * AC_ROWS / a.G, x, hi);
        att_range(a, cur.s, (cur.rt * AC_ROWS + rows_of() - 1) / a.G, lo, x);
    };
    auto place = [&](int row, int c) { return (c >> 3) * BLK + row * 128 + ((c ^ row) & 7) * 16; };  // 16-byte piece c

    if (warp < 8) {
        // ------------------------------------------------ softmax, one thread per row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int half = warp >> 2, r = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21), t_s = lanes + S_COL + half * 128,
                       t_o = lanes + O_COL + half * D;
        uint8_t* const q_s = smem + half * TILE;
        uint32_t s_ph = 0, o_ph = 0, h_ph = 0;
        bool dead = false;
        for (int item = 0; !dead && next_piece(); ++item) {
            const int rows = rows_of();
            const bool duo = rows <= 128;  // both halves hold the same rows and take the tiles in turn
            const int row0 = duo ? 0 : half * 128, steps = duo ? (cnt + 1 - half) / 2 : cnt;
            const int rr = cur.rt * AC_ROWS + row0 + r, i = rr / a.G, head = cur.h * a.G + rr % a.G;
            const bool mine = row0 + r < rows, busy = __any_sync(~0u, mine);  // a warp without rows only keeps step
            int lo = 0, hi = 0x7fffffff;  // (a lane without a row must not make its warp mask)
            if (mine) att_range(a, cur.s, i, lo, hi);
            const int pos = cur.s.p0 + i;
            const float ks = (F8 && a.k_scale) ? __ldg(a.k_scale + cur.h) : 1.f;
            const float vs = (F8 && a.v_scale) ? __ldg(a.v_scale + cur.h) : 1.f;
            const bool simple = MODE == 0 && a.scale * ks > 0.f;  // scores are S times a positive number
            const float slope = ((MODE & 1) && mine) ? __ldg(a.slopes + head) * LOG2E : 0.f;
            // ---- Q: this warp's 32 rows into the half's K-major operand tile, LPR lanes to a row.  The loops
            // that run once an item are kept short: unrolled, they cost more in instruction fetches.
            constexpr int LPR = D / 8, RPI = 32 / LPR;
            float unit = 1.f;
            {
                const int64_t off = mine ? (int64_t)(cur.s.t0 + i) * a.q_stride + head * D : -1;
                uint8_t* const q_w = q_s + (warp & 3) * 32 * 128;
#pragma unroll 1
                for (int n = 0; n < LPR; ++n) {
                    const int q = n * RPI + lane / LPR;
                    const int64_t o = __shfl_sync(~0u, off, q);
                    cp_async16(smem_u32(q_w + place(q, lane % LPR)), a.q + (o < 0 ? 0 : o) + (lane % LPR) * 8, o >= 0);
                }
                cp_async_commit();
                cp_async_wait<0>();
                if constexpr (F8) {  // the row's largest element to [2^14, 2^15), all of them to fp16
#pragma unroll 2
                    for (int n = 0; n < LPR; ++n) {
                        uint4* const at = reinterpret_cast<uint4*>(q_w + place(n * RPI + lane / LPR, lane % LPR));
                        const uint4 w = *at;
                        uint32_t x[4] = {w.x, w.y, w.z, w.w};
                        uint32_t top = 0;  // magnitudes of bf16 values compare as integers
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = max(top, max(x[e] << 16 & 0x7fffffffu, x[e] & 0x7fff0000u));
#pragma unroll
                        for (int d = 1; d < LPR; d <<= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
                        const int be = (int)(top >> 23);
                        const int e2 = be == 255 ? 0 : max(be - 127 - 14, -100);
                        const float down = __uint_as_float((uint32_t)(127 - e2) << 23), up = __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] = pack_f16x2(__uint_as_float(x[e] << 16) * down, __uint_as_float(x[e] & 0xffff0000u) * down);
                        *at = make_uint4(x[0], x[1], x[2], x[3]);
                        const float mine_up = __shfl_sync(~0u, up, (lane % RPI) * LPR);
                        if (lane / RPI == n) unit = mine_up;
                    }
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(qready);
            // (above zero where it multiplies hidden scores, -inf: queries of zeros under a scale of 2^-64 underflow it)
            const float rs0 = a.scale * ks * unit * LOG2E, rs = simple ? fmaxf(rs0, 1.17549435e-38f) : rs0;
            const AttCap cap(a.softcap);
            float m = -INFINITY, l = 0.f;
            for (int n = 0; n < steps; ++n) {
                const int j = duo ? 2 * n + half : n;
                if (!__all_sync(~0u, mbar_wait_fast(sfull + half, s_ph, 21, j))) { dead = true; break; }
                s_ph ^= 1;
                if (busy) {
                    tc_fence_after();
                    const int k0 = cur.lo + (cur.tile + j) * AC_TK;
                    const bool masked = __any_sync(~0u, k0 < lo || k0 > hi - AC_TK), edit = masked || !simple;
                    // (two forms of the same: 2,048 tokens with slopes at 64K take 1.39 ms in the first for e4m3, 1.47 in
                    // the second; for bf16 1.39 and 1.30)
                    const bool tilted = MODE == 1 && !masked && (F8 ? __all_sync(~0u, !mine || k0 + AC_TK - 1 <= pos)
                                                                    : !__any_sync(~0u, mine && k0 + AC_TK - 1 > pos));
                    // Scores that are not S times a number, or hidden ones, are put in S's place first; but a slope
                    // alone is linear in the column of a tile behind the row, and is added to the registers below.
                    uint32_t u[128];
                    auto load_s = [&] {
#pragma unroll
                        for (int g = 0; g < 4; ++g) tmem_ld32(t_s + g * 32, u + g * 32);
                        tmem_ld_wait();
#pragma unroll
                        for (int g = 0; g < 4; ++g) reg_tie32(u + g * 32);
                    };
                    bool capped = false;
                    if (MODE == 2 && !masked) {  // all scores well below the cap: a polynomial, no special functions
                        load_s();
                        float far[2] = {0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < 128; c += 2) {
                            far[0] = fmaxf(far[0], fabsf(__uint_as_float(u[c])));
                            far[1] = fmaxf(far[1], fabsf(__uint_as_float(u[c + 1])));
                        }
                        // u becomes S (1 + z q(z)), z = (S rs / cap)^2, still to be multiplied by rs
                        const float y = rs * cap.in;
                        capped = __all_sync(~0u, !mine || (rs > 0.f && fmaxf(far[0], far[1]) * y <= 0.7f));
                        if (capped) {
                            const float2 y2 = both(y), zero = both(0.f), one = both(1.f);
#pragma unroll
                            for (int c = 0; c < 128; c += 2) {
                                const float2 x = make_float2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), t = fma2(x, y2, zero),
                                             z = fma2(t, t, zero), r = fma2(x, fma2(z, ac_cap_poly2(z), one), zero);
                                u[c] = __float_as_uint(r.x);
                                u[c + 1] = __float_as_uint(r.y);
                            }
                        }
                    }
                    if (F8 && MODE == 1 ? !tilted : edit && !tilted && !capped) {
                        const int f = masked ? lo - k0 : -1024, e = masked ? hi - k0 : 1024;  // visible columns [f, e)
                        const float p0 = (float)(pos - k0);
#pragma unroll 1
                        for (int g = 0; g < 128; g += 16) {
                            uint32_t v[16];
                            tmem_ld16(t_s + g, v);
                            tmem_ld_wait16(v);
#pragma unroll
                            for (int c = 0; c < 16; c += 2) {
                                float2 x = make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1]));
                                if (!simple) {
                                    x = make_float2(x.x * rs, x.y * rs);
                                    if constexpr ((MODE & 2) != 0) x = cap(x);
                                    if constexpr ((MODE & 1) != 0) {
                                        x.x -= slope * fabsf(p0 - (float)(g + c));
                                        x.y -= slope * fabsf(p0 - (float)(g + c + 1));
                                    }
                                }
                                v[c] = g + c >= f && g + c < e ? __float_as_uint(x.x) : 0xff800000u;  // -inf
                                v[c + 1] = g + c + 1 >= f && g + c + 1 < e ? __float_as_uint(x.y) : 0xff800000u;
                            }
                            tmem_st16(t_s + g, v);
                        }
                        tmem_st_wait();
                    }
                    if (!capped) load_s();
                    if (tilted) {
                        // the bias from the column every 8 of them: a running sum over all drifts by 2^-19 of the bias
                        const float2 rs2 = both(rs), slope2 = both(slope), at0 = both(-slope * (float)(pos - k0)), step = both(2.f * slope);
                        float2 bias;
#pragma unroll
                        for (int c = 0; c < 128; c += 2) {
                            bias = c % 8 ? add2(bias, step) : fma2(make_float2((float)c, (float)(c + 1)), slope2, at0);
                            const float2 x = fma2(make_float2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), rs2, bias);
                            u[c] = __float_as_uint(x.x);
                            u[c + 1] = __float_as_uint(x.y);
                        }
                    }
                    float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 128; c += 2)
                        t4[(c >> 1) & 3] = fmaxf(t4[(c >> 1) & 3], fmaxf(__uint_as_float(u[c]), __uint_as_float(u[c + 1])));
                    const float mul = simple || capped ? rs : 1.f;
                    const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * mul;
                    const bool grew = top > m + GROW || (m == -INFINITY && top > m);
                    if (__any_sync(~0u, grew)) {
                        const float f = grew ? ex2(m - top) : 1.f;
                        if (grew) m = top;
                        l *= f;
                        if (n > 0) {  // O holds sums already
#pragma unroll 1
                            for (int c = 0; c < D; c += 8) {
                                uint32_t o[8];
                                tmem_ld8(t_o + c, o);
                                tmem_ld_wait();
                                reg_tie8(o);
#pragma unroll
                                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st8(t_o + c, o);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m - LIFT;
                    // Numerators, their sum unrounded, and their 16-bit form over S: bf16 (2^-8) beside bf16 values, since
                    // an MMA takes one type and fp16 lacks bf16's range; fp16 (2^-11) beside e4m3 ones, which it holds
                    // exactly.  A second 16-bit part would be half as many products again.
                    const float2 mul2 = make_float2(mul, mul), ref2 = make_float2(-ref, -ref);
                    float2 la = make_float2(0.f, 0.f), lb = la;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t p[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            float2 x = fma2(make_float2(__uint_as_float(u[g * 32 + 2 * c]), __uint_as_float(u[g * 32 + 2 * c + 1])), mul2, ref2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            if (c & 1) lb = add2(lb, x);
                            else la = add2(la, x);
                            p[c] = F8 ? pack_f16x2(x.x, x.y) : pack_bf16x2(x.x, x.y);
                        }
                        tmem_st16(t_s + g * 16, p);
                    }
                    la = add2(la, lb);
                    l += la.x + la.y;
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + half);
            }
            if (dead) break;
            // ---- the piece ends: the rows, or their partial sums
            if (!__all_sync(~0u, mbar_wait(ofull, o_ph, 22, item))) { dead = true; break; }
            o_ph ^= 1;
            tc_fence_after();
            const bool first = cur.tile == 0, last = cur.tile + cnt == cur.n, whole = first && last;
            const int slot = 2 * blockIdx.x + (first ? 1 : 0);
            // Two rounds of D / 2 columns.  A thread's columns are staged in its row of the (now free) Q tile,
            // so that the warp writes whole row pieces to memory; where both halves held the rows, the second
            // half's sums come over through its own Q tile, [column][row], and the first half adds them.
            const bool two = duo && cnt > 1;
            const int64_t row = (int64_t)(cur.s.t0 + i) * (a.Hk * a.G) + head;
            const int64_t prow = (int64_t)slot * AC_ROWS + row0 + r;
            const bool fix = odd[item & 7] == item + 1;
            float* const other = reinterpret_cast<float*>(smem + TILE);
            float f0 = 1.f, f1 = 0.f, f = 0.f;
#pragma unroll 1
            for (int c0 = 0; c0 < D && !dead; c0 += D / 2) {
                if (two) {
                    if (half == 1) {
                        if (busy) {
                            if (c0 == 0) half_ml[r] = make_float2(m, l);
#pragma unroll 1
                            for (int c = 0; c < D / 2; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(t_o + c0 + c, o);
                                tmem_ld_wait();
                                reg_tie32(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) other[(c + e) * 128 + r] = __uint_as_float(o[e]);
                            }
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(half_up);
                    } else if (!__all_sync(~0u, mbar_wait(half_up, h_ph, 31, item))) {
                        dead = true;
                        break;
                    }
                }
                if (busy && !(duo && half == 1)) {
                    if (c0 == 0) {
                        if (two && mine) {
                            const float2 o = half_ml[r];
                            const float mn = fmaxf(m, o.x);
                            f0 = m == mn ? 1.f : ex2(m - mn);
                            f1 = o.x == mn ? 1.f : ex2(o.x - mn);
                            m = mn;
                            l = l * f0 + o.y * f1;
                        }
                        f = !whole ? vs : l == 0.f ? 0.f : vs / l;
                    }
                    // FIX: non-finite values in masked tiles were taken out of the product; back to the rows that see them
                    auto columns = [&](auto fix_tag) {
                        constexpr bool FIX = decltype(fix_tag)::value;
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(t_o + c0 + c, o);
                            tmem_ld_wait16(o);
                            float x[16];
                            if (two) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(o[e]) * f0 + other[(c + e) * 128 + r] * f1;
                            } else {
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(o[e]);
                            }
                            if constexpr (FIX) {
                                int all_lo, all_hi;
                                seen_by_all(all_lo, all_hi);
                                for (int j = 0; j < cnt; ++j) {
                                    const int k0 = cur.lo + (cur.tile + j) * AC_TK;
                                    if (k0 >= all_lo && k0 + AC_TK <= all_hi) continue;
                                    for (int key = max(k0, lo); key < min(k0 + AC_TK, hi); ++key) {
                                        const int col = key / a.page_size, pg = __ldg(a.table + (int64_t)cur.b * a.width + col);
                                        if (pg < 0 || pg >= a.n_pages) continue;
                                        const uint8_t* vp = a.v + pg * a.page_b + (int64_t)(key - col * a.page_size) * a.token_b +
                                                            cur.h * a.head_b;
#pragma unroll
                                        for (int e = 0; e < 16; ++e) {
                                            float y;
                                            if constexpr (F8) y = half_bits_to_f32((uint16_t)e4m3x2_to_f16x2(vp[c0 + c + e]));
                                            else y = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(vp)[c0 + c + e]);
                                            if (!(fabsf(y) < INFINITY)) x[e] += y;
                                        }
                                    }
                                }
                            }
                            if (whole) {
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    *reinterpret_cast<uint4*>(q_s + place(r, c / 8 + e)) = make_uint4(
                                        pack_bf16x2(x[8 * e] * f, x[8 * e + 1] * f), pack_bf16x2(x[8 * e + 2] * f, x[8 * e + 3] * f),
                                        pack_bf16x2(x[8 * e + 4] * f, x[8 * e + 5] * f), pack_bf16x2(x[8 * e + 6] * f, x[8 * e + 7] * f));
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    *reinterpret_cast<float4*>(q_s + place(r, c / 4 + e)) =
                                        make_float4(x[4 * e] * f, x[4 * e + 1] * f, x[4 * e + 2] * f, x[4 * e + 3] * f);
                            }
                        }
                    };
                    if (__any_sync(~0u, fix && mine)) columns(std::true_type{});
                    else columns(std::false_type{});
                    __syncwarp();
                    const int wr = (warp & 3) * 32;  // the warp's rows, so many lanes to each
                    if (whole) {
                        constexpr int L = D / 16;
#pragma unroll 4
                        for (int n = 0; n < L; ++n) {
                            const int q = n * (32 / L) + lane / L;
                            const int64_t to = __shfl_sync(~0u, row, q);
                            if (row0 + wr + q < rows)
                                *reinterpret_cast<uint4*>(a.out + to * D + c0 + (lane % L) * 8) =
                                    *reinterpret_cast<const uint4*>(q_s + place(wr + q, lane % L));
                        }
                    } else {
                        constexpr int L = D / 8;
#pragma unroll 4
                        for (int n = 0; n < L; ++n) {
                            const int q = n * (32 / L) + lane / L;
                            if (row0 + wr + q < rows)
                                *reinterpret_cast<uint4*>(a.part + (prow - lane + q) * D + c0 + (lane % L) * 4) =
                                    *reinterpret_cast<const uint4*>(q_s + place(wr + q, lane % L));
                        }
                    }
                    __syncwarp();
                }
                if (two) {  // the second half's tile is free again once every warp of the first half has read it
                    __syncwarp();
                    if (half == 0 && lane == 0) mbar_arrive(half_read);
                    if (half == 1 && !__all_sync(~0u, mbar_wait(half_read, h_ph, 32, item))) { dead = true; break; }
                    h_ph ^= 1;
                }
            }
            if (dead) break;
            if (mine && !(duo && half == 1)) {
                if (!whole) a.ml[prow] = make_float2(m, l);
                else if (a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m - LIFT + log2f(l)) * 0.6931471805599453f;
            }
            if (first && !last && tid == 0) {  // the join starts from here
                const int parts = (rel + AC_OV + cur.n - 1) / share + 1;
                a.hdr[blockIdx.x] = make_int4(parts | rows << 16, cur.s.t0, cur.rt * AC_ROWS, cur.h);
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------ widening, cleaning, or the whole gather
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int t = tid - 256;
        constexpr int CHG = D * (F8 ? 1 : 2) / 16, STEP = 128 / CHG;  // 16-byte pieces of a cached row; rows a pass
        const int c = t % CHG, t_row = t / CHG;
        // two 16-bit values, non-finite ones set to zero; `note` 0: of a key that no row sees (never written, or
        // behind a window), which need not be added back
        auto clean2 = [&](uint32_t x, int note) {
            constexpr uint32_t EXP = F8 ? 0x7c00u : 0x7f80u;
            uint32_t keep = ~0u;
            if ((x & EXP) == EXP) keep &= 0xffff0000u;
            if ((x & EXP << 16) == EXP << 16) keep &= 0x0000ffffu;
            if (keep != ~0u && note) odd[(note - 1) & 7] = note;
            return x & keep;
        };
        // 16 e4m3 values into their two pieces of this thread's first row of a tile; its rows are STEP (a
        // multiple of 8) apart, so the others' places differ by a constant
        static_assert(!F8 || STEP % 8 == 0, "the swizzle repeats every 8 rows");
        const bool turn = D == 128 && (c & 4);  // the second block's lanes start with the other piece: no bank twice
        const int at0 = place(t_row, 2 * c + turn), at1 = place(t_row, 2 * c + 1 - turn);
        auto widen = [&](uint4 w, uint8_t* dst, bool clean, int note) {
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[2 * e] = e4m3x2_to_f16x2(x[e]);
                y[2 * e + 1] = e4m3x2_to_f16x2(x[e] >> 16);
            }
            if (clean) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = clean2(y[e], note);
            }
            const uint4 p0 = make_uint4(y[0], y[1], y[2], y[3]), p1 = make_uint4(y[4], y[5], y[6], y[7]);
            *reinterpret_cast<uint4*>(dst + at0) = turn ? p1 : p0;
            *reinterpret_cast<uint4*>(dst + at1) = turn ? p0 : p1;
        };
        auto clean_own = [&](uint8_t* dst, int seen0, int seen1, int item) {  // bf16: this thread's pieces of a tile, keys seen in [seen0, seen1)
#pragma unroll 1
            for (int row = t_row; row < AC_TK; row += STEP) {
                uint4* p = reinterpret_cast<uint4*>(dst + place(row, c));
                const uint4 w = *p;
                const int note = row >= seen0 && row < seen1 ? item + 1 : 0;
                const uint4 n = make_uint4(clean2(w.x, note), clean2(w.y, note), clean2(w.z, note), clean2(w.w, note));
                if (n.x != w.x || n.y != w.y || n.z != w.z || n.w != w.w) *p = n;
            }
        };
        int slot = 0, rslot = 0, item = 0;
        uint32_t ph = 0, rph = 0;
        auto step = [&] { if (++slot == NS) { slot = 0; ph ^= 1; } };
        bool ok = true;
        if (a.tma) {
            // e4m3: the four warps widen every tile together, in the ring's order; bf16: they watch the V tiles
            for (; ok && next_piece(); ++item) {
                int all_lo, all_hi;
                seen_by_all(all_lo, all_hi);
                for (int j = 0; j < cnt && ok; ++j) {
                    const int k0 = cur.lo + (cur.tile + j) * AC_TK;
                    const bool some_hidden = k0 < all_lo || k0 + AC_TK > all_hi;
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, step()) {
                        const bool masked = kv && some_hidden;
                        uint8_t* const dst = smem + C::OFF_RING + slot * TILE;
                        if constexpr (F8) {
                            ok = mbar_wait_fast(raw_full + rslot, rph, 23, rslot) && mbar_wait_fast(empty + slot, ph ^ 1, 24, slot);
                            if (!ok) break;
                            const uint8_t* const src = smem + C::OFF_RAW + rslot * C::RAW + t_row * D + c * 16;
                            if (masked) {
#pragma unroll 1
                                for (int n = 0; n < AC_TK / STEP; ++n) {
                                    const int key = k0 + t_row + n * STEP;
                                    widen(*reinterpret_cast<const uint4*>(src + n * STEP * D), dst + n * STEP * 128, true,
                                          key >= cur.first && key < cur.hi ? item + 1 : 0);
                                }
                            } else {
#pragma unroll 4
                                for (int n = 0; n < AC_TK / STEP; ++n)
                                    widen(*reinterpret_cast<const uint4*>(src + n * STEP * D), dst + n * STEP * 128, false, 0);
                            }
                            mbar_arrive(raw_empty + rslot);
                            fence_proxy_async_smem();
                            mbar_arrive(full + slot);
                            if (++rslot == NRAW) {
                                rslot = 0;
                                rph ^= 1;
                            }
                        } else if (kv) {  // every V tile passes through here, so that the phases cannot run apart
                            ok = mbar_wait_fast(full + slot, ph, 23, slot);
                            if (!ok) break;
                            if (masked) {
                                clean_own(dst, cur.first - k0, cur.hi - k0, item);
                                fence_proxy_async_smem();
                            }
                            mbar_arrive(cleaned + slot);
                        }
                    }
                }
            }
        } else {
            // rows gathered one by one: thread t looks up key t of a tile, one tile ahead
            int pg = 0, pg_off = 0, j = 0;
            bool pg_live = false;
            auto fetch = [&] {
                const int key = cur.lo + (cur.tile + j) * AC_TK + t;
                pg_live = key >= cur.first && key < cur.hi;
                if (pg_live) {
                    const int col = key / a.page_size;
                    pg_off = key - col * a.page_size;
                    pg = __ldg(a.table + (int64_t)cur.b * a.width + col);
                }
            };
            int all_lo = 0, all_hi = 0;
            bool more = next_piece();
            if (more) {
                seen_by_all(all_lo, all_hi);
                fetch();
            }
            for (int it = 0; more && ok; ++it) {
                int64_t* const of = offs + (it & 1) * AC_TK;
                int64_t o = -1;
                if (pg_live) {
                    if (pg >= 0 && pg < a.n_pages) o = pg * a.page_b + pg_off * a.token_b + cur.h * a.head_b;
                    else moe_set_status(MOE_ERR_SLOT);  // its keys read as zeros
                }
                of[t] = o;
                const int k0 = cur.lo + (cur.tile + j) * AC_TK, this_item = item;
                const bool masked = k0 < all_lo || k0 + AC_TK > all_hi;
                if (++j == cnt) {
                    j = 0;
                    more = next_piece();
                    ++item;
                    if (more) seen_by_all(all_lo, all_hi);
                }
                if (more) fetch();
                mbar_arrive(rows_up);
                ok = mbar_wait(rows_up, it & 1, 33, it);  // the 128 row offsets are there
                for (int kv = 0; kv < 2 && ok; ++kv, step()) {
                    ok = mbar_wait_fast(empty + slot, ph ^ 1, 24, slot);
                    if (!ok) break;
                    uint8_t* const dst = smem + C::OFF_RING + slot * TILE;
                    const uint8_t* const src = (kv ? a.v : a.k) + c * 16;
#pragma unroll 2
                    for (int row = t_row; row < AC_TK; row += STEP) {
                        const int64_t from = of[row];
                        if constexpr (F8)
                            widen(from >= 0 ? *reinterpret_cast<const uint4*>(src + from) : make_uint4(0, 0, 0, 0),
                                  dst + (row - t_row) * 128, kv && masked, this_item + 1);
                        else
                            cp_async16(smem_u32(dst + place(row, c)), src + (from < 0 ? 0 : from), from >= 0);
                    }
                    if constexpr (!F8) {
                        cp_async_commit();
                        cp_async_wait<0>();
                        if (kv && masked) clean_own(dst, 0, AC_TK, this_item);  // (a key that no row sees is a row of zeros)
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(full + slot);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 12 && elect_one()) {
            // -------------------------------------------- MMAs, one thread
            constexpr uint32_t ID_QK = ac_idesc(F8 ? 0 : 1, AC_TK, false), ID_PV = ac_idesc(F8 ? 0 : 1, D, true);
            const uint32_t sq = smem_u32(smem), ring = sq + C::OFF_RING;
            uint32_t q_ph = 0, o_ph = 0, p_ph[2] = {0, 0};
            uint64_t* const v_up = !F8 && a.tma ? cleaned : full;
            int ks = 0, vsl = 1;  // ring places of the next K and V tile, and their phases
            uint32_t k_ph = 0, v_ph = 0;
            bool ok = true;
            auto next2 = [&](int& s, uint32_t& ph) {
                s += 2;
                if (s >= NS) {
                    s -= NS;
                    ph ^= 1;
                }
            };
            for (int item = 0; ok && next_piece(); ++item) {
                const bool duo = rows_of() <= 128;
                const int steps = duo ? cnt : 2 * cnt;
                ok = mbar_wait(qready, q_ph, 26, item);
                q_ph ^= 1;
                tc_fence_after();
                for (int s = 0; s <= steps && ok; ++s) {
                    if (s < steps) {
                        const int h = s & 1;
                        if (duo || h == 0) ok = mbar_wait_fast(full + ks, k_ph, 25, ks);
                        if (!ok) break;
                        tc_fence_after();
                        // (descriptor addresses count in 16 bytes)
                        uint64_t da = make_sdesc_sw128(sq + h * TILE), db = make_sdesc_sw128(ring + ks * TILE);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_bf16(tmem + S_COL + h * 128, da + (k >> 2) * (BLK / 16) + (k & 3) * 2, db + (k >> 2) * (BLK / 16) + (k & 3) * 2, ID_QK, k > 0);
                        tc_commit(sfull + h);
                        if (duo || h == 1) {
                            tc_commit(empty + ks);
                            next2(ks, k_ph);
                        }
                    }
                    if (s > 0) {
                        const int h = (s - 1) & 1, j = duo ? s - 1 : (s - 1) >> 1;
                        if (duo || h == 0) ok = mbar_wait_fast(v_up + vsl, v_ph, 27, vsl);
                        ok = ok && mbar_wait_fast(pfull + h, p_ph[h], 29, h);
                        if (!ok) break;
                        p_ph[h] ^= 1;
                        tc_fence_after();
                        const bool add = duo ? j > 1 : j > 0;
                        uint64_t dv = make_sdesc_v(ring + vsl * TILE);
#pragma unroll
                        for (int k = 0; k < AC_TK / 16; ++k)
                            tc_mma_bf16_ts(tmem + O_COL + h * D, tmem + S_COL + h * 128 + k * 8, dv + k * 128, ID_PV, add || k > 0);
                        if (duo || h == 1) {
                            tc_commit(empty + vsl);
                            next2(vsl, v_ph);
                        }
                    }
                }
                tc_commit(ofull);
                if (!ok) mbar_wait(ofull, o_ph, 30, item);  // a wait expired: nothing in flight when TMEM is given back
                o_ph ^= 1;
            }
        } else if (warp == 13 && a.tma) {
            // -------------------------------------------- TMA loads, a lane per page of a tile
            const int ps = a.page_size, high = min(ps, AC_TK), np = AC_TK / high;  // tokens a box, boxes a tile
            int slot = 0;
            uint32_t ph = 1;
            constexpr int N = F8 ? NRAW : NS;
            uint64_t *const fb = F8 ? raw_full : full, *const eb = F8 ? raw_empty : empty;
            uint8_t* const base = smem + (F8 ? C::OFF_RAW : C::OFF_RING);
            constexpr uint32_t BYTES = F8 ? C::RAW : TILE;
            int pg = 0, issued = 0, j = 0;
            // page of box `lane`; wholly before the first visible key or past the last one no row reads it, and the
            // table may hold anything there (pages given back behind a window): none is looked up
            auto fetch = [&] {
                const int key = cur.lo + (cur.tile + j) * AC_TK + lane * high;
                pg = -1;
                if (lane < np && key + high > cur.first && key < cur.hi) {
                    pg = __ldg(a.table + (int64_t)cur.b * a.width + key / ps);
                    if (pg < 0 || pg >= a.n_pages) {
                        moe_set_status(MOE_ERR_SLOT);  // a box outside the cache reads as zeros
                        pg = a.n_pages;
                    }
                } else {
                    pg = a.n_pages;
                }
            };
            if (lane == 0) {
                tma_prefetch_desc(&tk);
                tma_prefetch_desc(&tv);
            }
            bool ok = true, more = next_piece();
            if (more) fetch();
            while (more && ok) {
                const int page = pg, h = cur.h, tok = (cur.lo + (cur.tile + j) * AC_TK) % ps;
                if (++j == cnt) {
                    j = 0;
                    more = next_piece();
                }
                if (more) fetch();
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    ok = __all_sync(~0u, mbar_wait_fast(eb + slot, ph, 23, slot));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(fb + slot, BYTES);
                    __syncwarp();
                    ++issued;
                    if (lane < np) {
                        uint8_t* const dst = base + slot * BYTES;
                        if constexpr (F8) {
                            tma_load_4d(dst + lane * high * D, kv ? &tv : &tk, fb + slot, 0, ps > AC_TK ? tok : 0, h, page);
                        } else {
#pragma unroll
                            for (int b = 0; b < D / 64; ++b)
                                tma_load_4d(dst + b * BLK + lane * high * 128, kv ? &tv : &tk, fb + slot, b * 64,
                                            ps > AC_TK ? tok : 0, h, page);
                        }
                    }
                    if (++slot == N) {
                        slot = 0;
                        ph ^= 1;
                    }
                }
            }
            // nothing in flight when the CTA's shared memory is given back: the MMAs wait for every tile, or,
            // after an expired wait, this warp for its last ones
            if (!ok)
                for (int g = max(0, issued - N); g < issued; ++g) mbar_wait(fb + g % N, (g / N) & 1, 34, g % N);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}
