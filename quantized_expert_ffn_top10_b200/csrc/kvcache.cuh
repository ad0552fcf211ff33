// The paged key-value cache: block tables and slots of a step's new tokens from
// the requests' lengths, and the per-head norm and rotation that write the new
// keys and values into their slots.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

// ---------------------------------------------------------------- block tables and slots

#define KM_THREADS 256

struct KvMapArgs {
    const int32_t *kv_len, *q_len, *free_pages;
    int B, page_size, n_free, width, T;
    int32_t *table, *kv_len_new, *cu, *position, *slot, *n_used;
};

// A step's bookkeeping in one launch: every CTA scans the B requests itself
// (two 64-bit sums, 8 B per request from L2), so no CTA waits for another, and
// the tokens and new table entries are spread over the grid.  Latency-bound:
// the scan and one binary search per token.  Request b owns pages
// [start_b, start_b + need_b) of the free list, start = exclusive sum of need;
// a token looks its page up in the table (older pages, which no CTA writes) or
// in the free list (new ones), never in an entry written by this launch.
__global__ void __launch_bounds__(KM_THREADS) k_kv_map(KvMapArgs a) {
    extern __shared__ int32_t km_s[];
    int32_t* cu = km_s;                // [B + 1] first token of each request
    int32_t* start = km_s + a.B + 1;   // [B + 1] first free-list entry of each request
    __shared__ long long wq[KM_THREADS / 32], wn[KM_THREADS / 32];
    __shared__ int s_used;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_used = 0;
    const int ipt = (a.B + KM_THREADS - 1) / KM_THREADS, b0 = min(a.B, tid * ipt), b1 = min(a.B, b0 + ipt);
    const long long cap = (long long)a.width * a.page_size;
    const int64_t ps = a.page_size;
    bool bad = false;
    auto lens = [&](int b, long long& old, long long& nw) {
        old = a.kv_len[b];
        nw = a.q_len[b];
        if (old < 0 || nw < 0) bad = true;
        old = max(old, 0LL);
        nw = max(nw, 0LL);
    };
    // pages a request asks for; none when its row has no room for them
    auto pages = [&](long long old, long long nw, bool& room) {
        room = old + nw <= cap && old + nw <= 0x7fffffffLL;
        return room ? (old + nw + ps - 1) / ps - (old + ps - 1) / ps : 0LL;
    };
    long long sq = 0, sn = 0;
    for (int b = b0; b < b1; ++b) {
        long long old, nw;
        bool room;
        lens(b, old, nw);
        sq += nw;
        sn += pages(old, nw, room);
    }
    long long iq = sq, in = sn;  // inclusive over the threads
    for (int d = 1; d < 32; d <<= 1) {
        const long long tq = __shfl_up_sync(~0u, iq, d), tn = __shfl_up_sync(~0u, in, d);
        if (lane >= d) { iq += tq; in += tn; }
    }
    if (lane == 31) { wq[warp] = iq; wn[warp] = in; }
    __syncthreads();
    long long eq = iq - sq, en = in - sn, allq = 0;
    for (int w = 0; w < KM_THREADS / 32; ++w) {
        if (w < warp) { eq += wq[w]; en += wn[w]; }
        allq += wq[w];
    }
    bool short_of_pages = false;
    int used = 0;
    for (int b = b0; b < b1; ++b) {
        long long old, nw;
        bool room;
        lens(b, old, nw);
        const long long need = pages(old, nw, room);
        const bool ok = room && (need == 0 || en + need <= a.n_free);
        cu[b] = (int32_t)min(eq, (long long)a.T);
        start[b] = ok ? (int32_t)min(en, 0x7fffffffLL) : -1 - (int32_t)min(en, 0x7ffffffeLL);  // negative: not granted
        if (ok) used = max(used, need ? (int)(en + need) : 0);
        else short_of_pages = true;
        if (blockIdx.x == 0) a.kv_len_new[b] = (int32_t)min(ok ? old + nw : old, 0x7fffffffLL);
        eq += nw;
        en += need;
    }
    if (used) atomicMax(&s_used, used);  // a maximum: the order of the atomics does not matter
    if (tid == 0) cu[a.B] = (int32_t)min(allq, (long long)a.T);
    if (blockIdx.x == 0) {
        if (bad || (tid == 0 && allq > a.T)) moe_set_status(MOE_ERR_RANGE);
        if (short_of_pages) moe_set_status(MOE_ERR_PAGES);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int b = tid; b <= a.B; b += KM_THREADS) a.cu[b] = cu[b];
        if (tid == 0) a.n_used[0] = s_used;
    }
    const int step = gridDim.x * KM_THREADS, at = blockIdx.x * KM_THREADS + tid;
    auto start_of = [&](int b) { return start[b] >= 0 ? start[b] : -1 - start[b]; };
    for (int e = at; e < s_used; e += step) {  // new table entries: the last request that starts at or before e
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start_of(mid) <= e) lo = mid;
            else hi = mid;
        }
        const long long have = (max((long long)a.kv_len[lo], 0LL) + ps - 1) / ps;
        a.table[(int64_t)lo * a.width + have + (e - start_of(lo))] = a.free_pages[e];
    }
    for (int t = at; t < a.T; t += step) {
        int32_t pos = 0, slot = -1;
        if (t < cu[a.B]) {
            int lo = 0, hi = a.B;  // the last request that starts at or before t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            const long long old = max((long long)a.kv_len[lo], 0LL), p = old + (t - cu[lo]);
            pos = (int32_t)min(p, 0x7fffffffLL);
            if (start[lo] >= 0) {
                const long long have = (old + ps - 1) / ps, col = p / ps;
                const int32_t page = col < have ? a.table[(int64_t)lo * a.width + col]
                                                : a.free_pages[start[lo] + (col - have)];
                const long long sl = (long long)page * ps + p % ps;
                if (page < 0 || sl > 0x7fffffffLL) moe_set_status(MOE_ERR_SLOT);
                else slot = (int32_t)sl;
            }
        }
        a.position[t] = pos;
        a.slot[t] = slot;
    }
}

// ---------------------------------------------------------------- norm, rotation, cache write

struct RopeArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, out_stride;  // elements from token to token
    uint16_t* q_out;
    const int32_t *position, *slot;
    const float *q_norm, *k_norm, *inv_freq, *k_scale, *v_scale;
    float eps, rot_scale;
    int T, Hq, Hk, rot, interleaved;
    uint8_t *k_cache, *v_cache;
    int64_t page_b, token_b, head_b;  // bytes
    int page_size;
    int64_t n_slots;
};

// Eight floats as e4m3, one rounding each, values beyond +-448 at the end of the range.
__device__ __forceinline__ uint2 pack_e4m3x8(const float* x) {
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        r[i] = lo | hi << 16;
    }
    return make_uint2(r[0], r[1]);
}

#define QR_UNROLL 3       // 32-byte pieces a thread has in flight
// Threads of a CTA at most.  Two such CTAs an SM bound the registers: 64 a thread at 512; 72 at 448, which the e4m3
// chunk kernel needs, and with which four of its usual CTAs of 224 threads fit (76, and three: 27.2 us for 8,192
// tokens instead of 23.6).
constexpr __host__ __device__ int qr_threads(bool e4m3, int tok) { return e4m3 && tok > 1 ? 448 : 512; }
#define QR_TOKENS 4       // tokens of a CTA on chunks

// One CTA per TOK tokens.  A head is D / 16 lanes of two 16-byte chunks, so a head
// never crosses a warp: the norm's sum is a shuffle over those lanes, and a lane
// takes the chunks whose elements turn together (8 i and 8 i + rot / 2 in the half
// layout), so the rotation needs no exchange.  The tokens' angles are computed
// once, a thread each, while the rows' loads are in flight: the turns
// position * f / 2 pi in fp64, their fraction to sincospi in fp32 (position * f
// itself passes 2^17, where fp32 would keep 2^-7 rad).  Everything between the
// load and the store is fp32; one rounding to bf16 or e4m3.  Bound by memory and
// instruction issue on chunks, by one load-to-store latency on windows.  Measured
// at 8,192 tokens of 16 + 2 x 2 heads of 128, 84 MB: 23.2 us (3.6 TB/s) with four
// tokens a CTA; 44 us with one token a CTA and partners 8 elements at a time by
// shuffle (shared memory and shuffles at 80% of their rate).
template <int D, bool E4M3, int TOK>
__global__ void __launch_bounds__(qr_threads(E4M3, TOK), 2) k_qk_norm_rope(RopeArgs a) {
    constexpr int L = D / 16;  // lanes per head
    __shared__ float4 cs[TOK][D / 4];  // cosines and sines, two pairs to an entry, [pairs of a lane / 2][lane]: no bank twice
    __shared__ int64_t s_place[TOK];   // of the token's slot in the cache, bytes; negative: nothing is written
    const int t0 = blockIdx.x * TOK, tid = threadIdx.x, nth = blockDim.x, half = a.rot / 2, turning = a.rot / 16;
    const int nch = (a.Hq + 2 * a.Hk) * L, ntok = min(TOK, a.T - t0), total = ntok * nch;
    auto token = [&](int i) {  // of piece i
        int k = 0;
#pragma unroll
        for (int j = 1; j < TOK; ++j) k += i >= j * nch;
        return k;
    };
    // element offsets of a lane's two chunks in its head
    const int l = tid % L;
    int d0 = l * 16, d1 = d0 + 8;
    if (!a.interleaved && l < turning) {
        d0 = l * 8;
        d1 = d0 + half;
    }
    const bool turns_here = l < turning;
    bool angles = false;
    for (int i0 = 0; i0 < total; i0 += nth * QR_UNROLL) {
        uint4 raw[QR_UNROLL][2];
#pragma unroll
        for (int u = 0; u < QR_UNROLL; ++u) {
            const int i = i0 + u * nth + tid, k = token(i), head = (i - k * nch) / L;
            const int64_t t = t0 + k;
            raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
            if (i < total) {
                const uint16_t* p = head < a.Hq ? a.q + t * a.q_stride + head * D
                                    : head < a.Hq + a.Hk ? a.k + t * a.k_stride + (head - a.Hq) * D
                                                         : a.v + t * a.v_stride + (head - a.Hq - a.Hk) * D;
                raw[u][0] = *reinterpret_cast<const uint4*>(p + d0);
                raw[u][1] = *reinterpret_cast<const uint4*>(p + d1);
            }
        }
        if (!angles) {
            if (nth - 1 - tid < ntok) {
                const int32_t slot = __ldg(a.slot + t0 + nth - 1 - tid);
                int64_t place = -1;  // a padding row
                if (slot >= a.n_slots) moe_set_status(MOE_ERR_SLOT);
                else if (slot >= 0) place = (int64_t)(slot / a.page_size) * a.page_b + (int64_t)(slot % a.page_size) * a.token_b;
                s_place[nth - 1 - tid] = place;
            }
            for (int i = tid; i < ntok * half; i += nth) {
                const int k = TOK == 1 ? 0 : i / half, f = i - k * half, e = f & 7;
                const double turns = (double)__ldg(a.position + t0 + k) * (double)__ldg(a.inv_freq + f) * 0.15915494309189535;
                float s, c;
                sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
                reinterpret_cast<float2*>(&cs[k][(e >> 1) * turning + (f >> 3)])[e & 1] = make_float2(c * a.rot_scale, s * a.rot_scale);
            }
            __syncthreads();
            angles = true;
        }
#pragma unroll
        for (int u = 0; u < QR_UNROLL; ++u) {
            const int i = i0 + u * nth + tid, k = token(i), head = (i - k * nch) / L;
            if (i0 + u * nth + (tid & ~31) >= total) break;  // a warp without work
            const int64_t t = t0 + k;
            const bool is_q = head < a.Hq, is_v = head >= a.Hq + a.Hk;
            float x[16];
            const uint32_t w[8] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w,
                                   raw[u][1].x, raw[u][1].y, raw[u][1].z, raw[u][1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[2 * e] = __uint_as_float(w[e] << 16);
                x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
            const float* nw = is_q ? a.q_norm : is_v ? nullptr : a.k_norm;
            if (a.q_norm || a.k_norm) {
                float ss = 0.f, s2 = 0.f;
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    ss = fmaf(x[e], x[e], ss);
                    s2 = fmaf(x[e + 1], x[e + 1], s2);
                }
                ss += s2;
#pragma unroll
                for (int m = 1; m < L; m <<= 1) ss += __shfl_xor_sync(~0u, ss, m);
                if (nw) {
                    const float r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 n = __ldg(reinterpret_cast<const float4*>(nw + (q < 2 ? d0 : d1)) + (q & 1));
                        x[4 * q] *= r * n.x;
                        x[4 * q + 1] *= r * n.y;
                        x[4 * q + 2] *= r * n.z;
                        x[4 * q + 3] *= r * n.w;
                    }
                }
            }
            if (turns_here && !is_v) {
                auto turn = [](float& p, float& n, float c, float s) {
                    const float q = p * c - n * s;
                    n = n * c + p * s;
                    p = q;
                };
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // pairs 2e and 2e + 1 of this lane
                    const float4 r = cs[k][e * turning + l];
                    if (a.interleaved) {
                        turn(x[4 * e], x[4 * e + 1], r.x, r.y);
                        turn(x[4 * e + 2], x[4 * e + 3], r.z, r.w);
                    } else {
                        turn(x[2 * e], x[8 + 2 * e], r.x, r.y);
                        turn(x[2 * e + 1], x[8 + 2 * e + 1], r.z, r.w);
                    }
                }
            }
            const int64_t place = s_place[k];
            if (i >= total || place < 0) continue;
            if (is_q || !E4M3) {
                uint16_t* p = is_q ? a.q_out + t * a.out_stride + head * D
                                   : reinterpret_cast<uint16_t*>(is_v ? a.v_cache + place + (head - a.Hq - a.Hk) * a.head_b
                                                                      : a.k_cache + place + (head - a.Hq) * a.head_b);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    *reinterpret_cast<uint4*>(p + (c ? d1 : d0)) =
                        make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]), pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                                   pack_bf16x2(x[8 * c + 4], x[8 * c + 5]), pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
            } else {
                const int h = is_v ? head - a.Hq - a.Hk : head - a.Hq;
                const float* sc = is_v ? a.v_scale : a.k_scale;
                if (sc) {
                    // The correctly rounded quotient: times 1 / scale alone, ties between two codes can fall to the
                    // other one.  q0 + (x - q0 s) r, r = 1 / s correctly rounded (Markstein), both scaled by a power
                    // of two that keeps the products in range; q0 as it is where it saturates anyway (infinities).
                    float s = __ldg(sc + h);
                    const float k = fabsf(s) < 0x1p-60f ? 0x1p64f : fabsf(s) > 0x1p60f ? 0x1p-64f : 1.f;
                    s *= k;
                    const float r = 1.f / s;
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 v = fma2(make_float2(x[e], x[e + 1]), both(k), both(0.f)), q0 = fma2(v, both(r), both(0.f)),
                                     q = fma2(fma2(q0, both(-s), v), both(r), q0);
                        x[e] = fabsf(q0.x) < 512.f ? q.x : q0.x;
                        x[e + 1] = fabsf(q0.y) < 512.f ? q.y : q0.y;
                    }
                }
                uint8_t* p = (is_v ? a.v_cache : a.k_cache) + place + h * a.head_b;
                *reinterpret_cast<uint2*>(p + d0) = pack_e4m3x8(x);
                *reinterpret_cast<uint2*>(p + d1) = pack_e4m3x8(x + 8);
            }
        }
    }
}
