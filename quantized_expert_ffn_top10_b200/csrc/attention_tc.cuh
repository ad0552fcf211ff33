// Chunk attention on the 5th-generation tensor cores: row tiles of 2 x 128 rows
// (attention.cuh has the formulas, the items and the deal).
//
// Per key tile of 128 and half h of the rows: S_h = Q_h K^T (tcgen05.mma, both
// operands in shared memory, fp32 in TMEM), numerators P_h = exp2(S_h - m) by
// 128 threads, one row each, written over S_h in TMEM as 16-bit, and O_h += P_h V
// (A from TMEM, V as stored: keys x dims, an MN-major B operand).  The two halves
// alternate, so the tensor cores work on one while the other is in its softmax:
// issue order QK0(j), PV1(j-1), QK1(j), PV0(j), ...  A commit covers everything
// issued before it, so S_h(j) being ready also says that PV_h(j-1) is done, and
// the softmax threads may rescale O_h in place.  They do so only when a row's
// maximum has grown by more than 2^8 since its reference was taken: numerators
// stay below 2^8 (2^14 in fp16), which costs no precision, and after the first
// tiles it hardly ever happens.
//
// Roles (16 warps): 0-3 and 4-7 the softmax of the two halves, 8-11 the loads
// (rows gathered through the block table, any page size and strides), 12 the
// MMAs.  e4m3 rows are widened to fp16 on the way into shared memory, exactly;
// the queries are then scaled per row by a power of two, as in the row kernel.
#pragma once

#include "attention.cuh"

#define AC_THREADS 512
#define AC_ROWS 256
#define AC_TK 128

template <int D>
struct AcCfg {
    static constexpr int TILE = 128 * D * 2;                  // one 16-bit operand tile: a half of Q, K or V
    static constexpr int NS = D == 128 ? 4 : 8;               // ring of K and V tiles: K0 V0 K1 V1 ...
    static constexpr int OFF_RING = 2 * TILE, OFF_ROW = OFF_RING + NS * TILE;
    static constexpr int OFF_BAR = OFF_ROW + 2 * AC_TK * 8;
    static constexpr int SMEM = OFF_BAR + 256 + 1024;         // and room to align to 1024 bytes
};

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
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// no use of these registers is scheduled before this point (after a wait for the loads)
__device__ __forceinline__ void reg_tie32(uint32_t* r) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                          "+r"(r[i + 6]), "+r"(r[i + 7])::"memory");
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

template <int D, bool F8>
__global__ void __launch_bounds__(AC_THREADS, 1) k_attn_chunk(const AttnArgs a) {
    using C = AcCfg<D>;
    constexpr int TILE = C::TILE, NS = C::NS, BLK = AC_TK * 128;  // a 64-column block of a tile
    constexpr float LOG2E = 1.4426950408889634f, LIFT = F8 ? 6.f : 0.f, GROW = 8.f;
    constexpr uint32_t S_COL = 0, O_COL = 256;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    int64_t* const offs = reinterpret_cast<int64_t*>(smem + C::OFF_ROW);
    uint64_t* const bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t *const full = bar, *const empty = bar + NS, *const sfull = bar + 2 * NS, *const pfull = sfull + 2,
             *const qready = pfull + 2, *const ofull = qready + 1;
    uint32_t* const tm = reinterpret_cast<uint32_t*>(ofull + 1);
    volatile int* const odd = reinterpret_cast<int*>(tm + 2);  // [8]: 1 + the item whose masked tiles held non-finite values
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    AttCur cur;
    int64_t w0, per, total;
    att_deal<AC_ROWS, AC_TK, AC_THREADS>(a, reinterpret_cast<int*>(smem), reinterpret_cast<int64_t*>(smem + C::OFF_ROW), cur,
                                         w0, per, total);
    const int my = (int)max((int64_t)0, min(per, total - w0));
    if (tid == 0) a.hdr[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (my == 0) return;
    __syncthreads();  // the scan's shared memory is free
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, 128);
            mbar_init(empty + i, 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(sfull + h, 1);
            mbar_init(pfull + h, 4);
        }
        mbar_init(qready, 8);
        mbar_init(ofull, 1);
        fence_mbar_init();
        for (int i = 0; i < 8; ++i) odd[i] = 0;
    }
    if (warp == 12) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm;

    // this CTA's piece of the item at `cur`: tiles [cur.tile, cur.tile + n)
    auto piece = [&](int it) { return min(cur.n - cur.tile, my - it); };
    auto halves = [&] { return cur.s.n * a.G - cur.rt * AC_ROWS > 128 ? 2 : 1; };
    auto leave = [&](int n) {  // past the piece
        cur.tile += n - 1;
        att_next<AC_ROWS, AC_TK>(a, cur);
    };

    if (warp < 8) {
        // ------------------------------------------------ softmax, one thread per row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int half = warp >> 2, r = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21), t_s = lanes + S_COL + half * 128,
                       t_o = lanes + O_COL + half * D;
        uint8_t* const q_s = smem + half * TILE;
        uint32_t s_ph = 0, o_ph = 0;
        bool dead = false;
        for (int it = 0, item = 0; it < my && !dead; ++item) {
            const int cnt = piece(it);
            const bool live = half < halves();
            const int rows = min(AC_ROWS, cur.s.n * a.G - cur.rt * AC_ROWS);
            const int rr = cur.rt * AC_ROWS + half * 128 + r, i = rr / a.G, head = cur.h * a.G + rr % a.G;
            const bool mine = half * 128 + r < rows;
            int lo = 0, hi = 0;
            if (mine) att_range(a, cur.s, i, lo, hi);
            const int pos = cur.s.kv - cur.s.n + i;
            const float ks = (F8 && a.k_scale) ? __ldg(a.k_scale + cur.h) : 1.f;
            const float vs = (F8 && a.v_scale) ? __ldg(a.v_scale + cur.h) : 1.f;
            const bool simple = a.softcap == 0.f && !a.slopes && a.scale * ks > 0.f;  // scores are S times a positive number
            const float slope = (a.slopes && mine) ? __ldg(a.slopes + head) * LOG2E : 0.f;
            // ---- Q: this thread's row into the K-major operand tile
            float unit = 1.f;
            if (live) {
                const uint4* qp = reinterpret_cast<const uint4*>(a.q + (int64_t)(cur.s.t0 + i) * a.q_stride + head * D);
                uint4 w[D / 8];
#pragma unroll
                for (int c = 0; c < D / 8; ++c) w[c] = mine ? qp[c] : make_uint4(0, 0, 0, 0);
                if constexpr (F8) {
                    float top = 0.f;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xffff0000u))));
                    }
                    const int be = (int)(__float_as_uint(top) >> 23);
                    const int e2 = be == 255 ? 0 : max(be - 127 - 14, -100);
                    const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
                    unit = __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] = pack_f16x2(__uint_as_float(x[e] << 16) * down, __uint_as_float(x[e] & 0xffff0000u) * down);
                        w[c] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    *reinterpret_cast<uint4*>(q_s + (c >> 3) * BLK + r * 128 + ((c ^ r) & 7) * 16) = w[c];
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(qready);
            const float rs = a.scale * ks * unit * (a.softcap > 0.f ? 1.f : LOG2E);
            float m = -INFINITY, l = 0.f;
            for (int j = 0; live && j < cnt; ++j) {
                if (!__all_sync(~0u, mbar_wait_fast(sfull + half, s_ph, 21, j))) { dead = true; break; }
                s_ph ^= 1;
                tc_fence_after();
                uint32_t u[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_s + c * 32, u + c * 32);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) reg_tie32(u + c * 32);
                const int k0 = cur.lo + (cur.tile + j) * AC_TK;
                float mul = rs;
                if (!simple) {
                    mul = 1.f;
#pragma unroll
                    for (int c = 0; c < 128; ++c) {
                        float x = __uint_as_float(u[c]) * rs;
                        if (a.softcap > 0.f) {  // cap tanh(x / cap), tanh y = 1 - 2 / (1 + e^2y)
                            const float y = ex2(x * (2.f * LOG2E) / a.softcap);
                            x = (a.softcap * LOG2E) * (1.f - __fdividef(2.f, 1.f + y));
                        }
                        if (a.slopes) x -= slope * fabsf((float)(pos - k0 - c));
                        u[c] = __float_as_uint(x);
                    }
                }
                if (__any_sync(~0u, k0 < lo || k0 + AC_TK > hi)) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (k0 + c < lo || k0 + c >= hi) u[c] = 0xff800000u;  // -inf
                }
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 128; ++c) top = fmaxf(top, __uint_as_float(u[c]));
                top *= mul;
                const bool grew = top > m + GROW || (m == -INFINITY && top > m);
                if (__any_sync(~0u, grew)) {
                    const float f = grew ? ex2(m - top) : 1.f;
                    if (grew) m = top;
                    l *= f;
                    if (j > 0) {  // O holds sums already
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(t_o + c, o);
                            tmem_ld_wait();
                            reg_tie32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(t_o + c, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m - LIFT;
                // numerators, their sum unrounded, and their 16-bit form over S
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    uint32_t p[32];
                    float l0 = 0.f, l1 = 0.f;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float x0 = ex2(fmaf(__uint_as_float(u[h2 * 64 + 2 * c]), mul, -ref));
                        const float x1 = ex2(fmaf(__uint_as_float(u[h2 * 64 + 2 * c + 1]), mul, -ref));
                        l0 += x0;
                        l1 += x1;
                        p[c] = F8 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
                    }
                    l += l0 + l1;
                    tmem_st32(t_s + h2 * 32, p);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + half);
            }
            if (dead) break;
            // ---- the piece ends: the rows, or their partial sums
            if (!__all_sync(~0u, mbar_wait(ofull, o_ph, 22, item))) { dead = true; break; }
            o_ph ^= 1;
            tc_fence_after();
            const int64_t first = w0 + it - cur.tile;
            const bool last = cur.tile + cnt == cur.n, whole = first >= w0 && last;
            const int slot = 2 * blockIdx.x + (first >= w0 ? 1 : 0);
            if (live) {
                const int64_t row = (int64_t)(cur.s.t0 + i) * (a.Hk * a.G) + head;
                const int64_t prow = (int64_t)slot * AC_ROWS + half * 128 + r;
                const float f = !whole ? vs : l == 0.f ? 0.f : vs / l;
                const bool fix = odd[item & 7] == item + 1;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(t_o + c, o);
                    tmem_ld_wait();
                    reg_tie32(o);
                    if (fix && mine) {
                        // non-finite values in a masked tile were taken out of the product: back to the rows that see them
                        int all_lo, all_hi, x;
                        att_range(a, cur.s, cur.rt * AC_ROWS / a.G, x, all_hi);
                        att_range(a, cur.s, (cur.rt * AC_ROWS + rows - 1) / a.G, all_lo, x);
                        for (int j = 0; j < cnt; ++j) {
                            const int k0 = cur.lo + (cur.tile + j) * AC_TK;
                            if (k0 >= all_lo && k0 + AC_TK <= all_hi) continue;
                            for (int key = max(k0, lo); key < min(k0 + AC_TK, hi); ++key) {
                                const int col = key / a.page_size, pg = __ldg(a.table + (int64_t)cur.b * a.width + col);
                                if (pg < 0 || pg >= a.n_pages) continue;
                                const uint8_t* vp = a.v + pg * a.page_b + (int64_t)(key - col * a.page_size) * a.token_b +
                                                    cur.h * a.head_b;
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    float y;
                                    if constexpr (F8) y = half_bits_to_f32((uint16_t)e4m3x2_to_f16x2(vp[c + e]));
                                    else y = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(vp)[c + e]);
                                    if (!(fabsf(y) < INFINITY)) o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
                                }
                            }
                        }
                    }
                    if (mine) {
                        if (whole) {
                            uint4* op = reinterpret_cast<uint4*>(a.out + row * D + c);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t y[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    y[z] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * z]) * f, __uint_as_float(o[8 * e + 2 * z + 1]) * f);
                                op[e] = make_uint4(y[0], y[1], y[2], y[3]);
                            }
                        } else {
                            float4* pp = reinterpret_cast<float4*>(a.part + prow * D + c);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                pp[e] = make_float4(__uint_as_float(o[4 * e]) * f, __uint_as_float(o[4 * e + 1]) * f,
                                                    __uint_as_float(o[4 * e + 2]) * f, __uint_as_float(o[4 * e + 3]) * f);
                        }
                    }
                }
                if (mine) {
                    if (!whole) a.ml[prow] = make_float2(m, l);
                    else if (a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m - LIFT + log2f(l)) * 0.6931471805599453f;
                }
            }
            it += cnt;
            if (it == my && tid == 0) {
                const int parts = !last && first >= w0 ? (int)((first + cur.n - 1) / per - blockIdx.x) + 1 : 0;
                a.hdr[blockIdx.x] = make_int4(parts, cur.s.t0, cur.rt * AC_ROWS, cur.h);
                a.hdr_rows[blockIdx.x] = rows;
            }
            if (it < my) leave(cnt);
        }
    } else if (warp < 12) {
        // ------------------------------------------------ loads
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        const int t = tid - 256;  // and the key of a tile this thread looks up
        constexpr int CHG = D * (F8 ? 1 : 2) / 16;  // 16-byte pieces of a cached row
        int pg = 0, pg_off = 0;
        bool pg_live = false;
        auto fetch = [&] {
            const int key = cur.lo + cur.tile * AC_TK + t;
            pg_live = key < cur.hi;
            if (pg_live) {
                const int col = key / a.page_size;
                pg_off = key - col * a.page_size;
                pg = __ldg(a.table + (int64_t)cur.b * a.width + col);
            }
        };
        // where piece c of row `row` goes in a tile (16-bit elements): 64-column blocks of swizzled 128-byte rows
        auto place = [&](int row, int c) { return (c >> 3) * BLK + row * 128 + ((c ^ row) & 7) * 16; };
        auto copy = [&](const uint8_t* src, const int64_t* of, uint32_t dst_a, uint8_t* dst, bool clean, int item) {
            (void)dst;
            if constexpr (!F8) {
                const int c = t % CHG;
#pragma unroll 8
                for (int row = t / CHG; row < AC_TK; row += 128 / CHG) {
                    const int64_t o = of[row];
                    cp_async16(dst_a + place(row, c), src + (o < 0 ? 0 : o) + c * 16, o >= 0);
                }
                cp_async_commit();
            } else {
                const int c = t % CHG;
                constexpr int NB = AC_TK * CHG / 128 > 8 ? 8 : AC_TK * CHG / 128;
#pragma unroll 1
                for (int r0 = t / CHG; r0 < AC_TK; r0 += NB * (128 / CHG)) {
                    uint4 w[NB];
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const int64_t o = of[r0 + n * (128 / CHG)];
                        w[n] = make_uint4(0, 0, 0, 0);
                        if (o >= 0) w[n] = *reinterpret_cast<const uint4*>(src + o + c * 16);
                    }
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const int row = r0 + n * (128 / CHG);
                        const uint32_t x[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
                        uint32_t y[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            y[2 * e] = e4m3x2_to_f16x2(x[e]);
                            y[2 * e + 1] = e4m3x2_to_f16x2(x[e] >> 16);
                        }
                        if (clean) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                uint32_t keep = ~0u;
                                if ((y[e] & 0x7c00u) == 0x7c00u) keep &= 0xffff0000u;
                                if ((y[e] & 0x7c000000u) == 0x7c000000u) keep &= 0x0000ffffu;
                                if (keep != ~0u) odd[item & 7] = item + 1;
                                y[e] &= keep;
                            }
                        }
                        *reinterpret_cast<uint4*>(dst + place(row, 2 * c)) = make_uint4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<uint4*>(dst + place(row, 2 * c + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
                    }
                }
            }
        };
        // bf16: this thread's pieces of a V tile with masked places, non-finite values taken out
        auto clean_own = [&](uint8_t* dst, int item) {
            const int c = t % CHG;
#pragma unroll 1
            for (int row = t / CHG; row < AC_TK; row += 128 / CHG) {
                uint32_t* p = reinterpret_cast<uint32_t*>(dst + place(row, c));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t x = p[e];
                    uint32_t keep = ~0u;
                    if ((x & 0x7f80u) == 0x7f80u) keep &= 0xffff0000u;
                    if ((x & 0x7f800000u) == 0x7f800000u) keep &= 0x0000ffffu;
                    if (keep != ~0u) {
                        odd[item & 7] = item + 1;
                        p[e] = x & keep;
                    }
                }
            }
        };
        int slot = 0, item = 0, v_item = 0;
        uint32_t ph = 1;  // a fresh ring is empty
        uint8_t* v_dst = nullptr;
        bool v_clean = false, ok = true;
        int all_lo = 0, all_hi = 0;
        bool entered = false;
        fetch();
        for (int it = 0; it < my; ++it) {
            if (!entered) {
                const int rows = min(AC_ROWS, cur.s.n * a.G - cur.rt * AC_ROWS);
                int x;
                att_range(a, cur.s, cur.rt * AC_ROWS / a.G, x, all_hi);
                att_range(a, cur.s, (cur.rt * AC_ROWS + rows - 1) / a.G, all_lo, x);
                entered = true;
            }
            int64_t* of = offs + (it & 1) * AC_TK;
            int64_t o = -1;
            if (pg_live) {
                if (pg >= 0 && pg < a.n_pages) o = pg * a.page_b + pg_off * a.token_b + cur.h * a.head_b;
                else moe_set_status(MOE_ERR_SLOT);  // its keys read as zeros
            }
            of[t] = o;
            const int k0 = cur.lo + cur.tile * AC_TK, this_item = item;
            const bool masked = k0 < all_lo || k0 + AC_TK > all_hi;
            if (it + 1 < my) {
                if (cur.tile + 1 == cur.n) {
                    ++item;
                    entered = false;
                }
                att_next<AC_ROWS, AC_TK>(a, cur);
                fetch();
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");  // the 128 row offsets are there
            for (int kv = 0; kv < 2; ++kv) {
                if (!mbar_wait_fast(empty + slot, ph, 23, slot)) { ok = false; break; }
                uint8_t* dst = smem + C::OFF_RING + slot * TILE;
                copy(kv ? a.v : a.k, of, smem_u32(dst), dst, kv && masked, this_item);
                if constexpr (F8) {
                    fence_proxy_async_smem();
                    mbar_arrive(full + slot);
                } else if (it > 0 || kv > 0) {  // the tile before this one has landed meanwhile
                    cp_async_wait<1>();
                    if (!kv && v_clean) clean_own(v_dst, v_item);
                    fence_proxy_async_smem();
                    mbar_arrive(full + (slot + NS - 1) % NS);
                }
                if (kv) {
                    v_dst = dst;
                    v_clean = masked;
                    v_item = this_item;
                }
                if (++slot == NS) {
                    slot = 0;
                    ph ^= 1;
                }
            }
            if (!ok) break;
        }
        if constexpr (!F8) {
            cp_async_wait<0>();
            if (ok) {
                if (v_clean) clean_own(v_dst, v_item);
                fence_proxy_async_smem();
                mbar_arrive(full + (slot + NS - 1) % NS);
            }
        }
    } else {
        // ------------------------------------------------ MMAs, one thread
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 12 && lane == 0) {
            constexpr uint32_t ID_QK = ac_idesc(F8 ? 0 : 1, AC_TK, false), ID_PV = ac_idesc(F8 ? 0 : 1, D, true);
            const uint32_t sq = smem_u32(smem), ring = sq + C::OFF_RING;
            uint32_t full_ph = 0, q_ph = 0, o_ph = 0, p_ph[2] = {0, 0};
            int slot = 0;
            bool ok = true;
            auto wait_full = [&](int s, uint32_t ph) { ok = ok && mbar_wait_fast(full + s, ph, 24, s); };
            auto wait_p = [&](int h) {
                ok = ok && mbar_wait_fast(pfull + h, p_ph[h], 25, h);
                p_ph[h] ^= 1;
                tc_fence_after();
            };
            auto qk = [&](int h, int s) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma_bf16(tmem + S_COL + h * 128, make_sdesc_sw128(sq + h * TILE + (k >> 2) * BLK + (k & 3) * 32),
                                make_sdesc_sw128(ring + s * TILE + (k >> 2) * BLK + (k & 3) * 32), ID_QK, k > 0);
                tc_commit(sfull + h);
            };
            auto pv = [&](int h, int s, bool add) {
#pragma unroll
                for (int k = 0; k < AC_TK / 16; ++k)
                    tc_mma_bf16_ts(tmem + O_COL + h * D, tmem + S_COL + h * 128 + k * 8,
                                   make_sdesc_v(ring + s * TILE + k * 2048), ID_PV, add || k > 0);
            };
            for (int it = 0; it < my && ok;) {
                const int cnt = piece(it), nh = halves();
                ok = mbar_wait(qready, q_ph, 26, it);
                q_ph ^= 1;
                tc_fence_after();
                for (int j = 0; j < cnt && ok; ++j) {
                    const int ks = slot, vsl = slot + 1, pv_prev = (slot + NS - 1) % NS;
                    wait_full(ks, full_ph);
                    if (!ok) break;
                    qk(0, ks);
                    if (nh == 2) {
                        if (j > 0) {
                            wait_p(1);
                            if (!ok) break;
                            pv(1, pv_prev, j > 1);
                            tc_commit(empty + pv_prev);
                        }
                        qk(1, ks);
                    }
                    tc_commit(empty + ks);
                    wait_full(vsl, full_ph);
                    wait_p(0);
                    if (!ok) break;
                    pv(0, vsl, j > 0);
                    if (nh == 1) tc_commit(empty + vsl);
                    slot += 2;
                    if (slot == NS) {
                        slot = 0;
                        full_ph ^= 1;
                    }
                }
                if (ok && nh == 2) {
                    const int pv_prev = (slot + NS - 1) % NS;
                    wait_p(1);
                    if (ok) {
                        pv(1, pv_prev, cnt > 1);
                        tc_commit(empty + pv_prev);
                    }
                }
                tc_commit(ofull);
                if (!ok) mbar_wait(ofull, o_ph, 27, it);  // a wait expired: nothing in flight when TMEM is given back
                o_ph ^= 1;
                it += cnt;
                if (it < my) leave(cnt);
            }
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
