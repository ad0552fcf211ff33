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
__device__ __forceinline__ uint2 pack_e4m3x8(const float (&x)[8]) {
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        r[i] = lo | hi << 16;
    }
    return make_uint2(r[0], r[1]);
}

#define QR_THREADS 160
#define QR_UNROLL 2

// One CTA per token.  A head is D / 8 lanes of 16 bytes, so a head never
// crosses a warp: the norm's sum is a shuffle over those lanes and the half
// layout's partner element sits rot / 16 lanes away.  The token's angles are
// computed once, by the first rot / 2 threads, while the row's loads are in
// flight: the turns position * f / 2 pi in fp64, their fraction to sincospi in
// fp32 (position * f itself passes 2^17, where fp32 would keep 2^-7 rad).
// Everything between the load and the store is fp32; one rounding to bf16 or
// e4m3.  Bound by memory on chunks, by one load-to-store latency on windows.
template <int D, bool E4M3>
__global__ void __launch_bounds__(QR_THREADS) k_qk_norm_rope(RopeArgs a) {
    constexpr int L = D / 8;  // lanes per head
    __shared__ float2 cs[D / 2];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int32_t slot = a.slot[t];
    if (slot < 0) return;  // a padding row: nothing of it is read or written
    if (slot >= a.n_slots) {
        if (tid == 0) moe_set_status(MOE_ERR_SLOT);
        return;
    }
    const int nch = (a.Hq + 2 * a.Hk) * L;
    const int64_t place = (int64_t)(slot / a.page_size) * a.page_b + (int64_t)(slot % a.page_size) * a.token_b;
    bool angles = false;
    for (int c0 = 0; c0 < nch; c0 += QR_THREADS * QR_UNROLL) {
        uint4 raw[QR_UNROLL];
#pragma unroll
        for (int u = 0; u < QR_UNROLL; ++u) {
            const int c = c0 + u * QR_THREADS + tid, head = c / L, d = (c % L) * 8;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (c < nch) {
                const uint16_t* p = head < a.Hq ? a.q + t * a.q_stride + head * D
                                    : head < a.Hq + a.Hk ? a.k + t * a.k_stride + (head - a.Hq) * D
                                                         : a.v + t * a.v_stride + (head - a.Hq - a.Hk) * D;
                raw[u] = *reinterpret_cast<const uint4*>(p + d);
            }
        }
        if (!angles) {
            if (tid < a.rot / 2) {
                const double turns = (double)a.position[t] * (double)a.inv_freq[tid] * 0.15915494309189535;
                float s, c;
                sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
                cs[tid] = make_float2(c * a.rot_scale, s * a.rot_scale);
            }
            __syncthreads();
            angles = true;
        }
#pragma unroll
        for (int u = 0; u < QR_UNROLL; ++u) {
            const int c = c0 + u * QR_THREADS + tid, head = c / L, d = (c % L) * 8;
            if (c0 + u * QR_THREADS + (tid & ~31) >= nch) continue;  // a warp without work
            const bool is_q = head < a.Hq, is_v = head >= a.Hq + a.Hk;
            float x[8];
            const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
            const float* nw = is_q ? a.q_norm : is_v ? nullptr : a.k_norm;
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int m = 1; m < L; m <<= 1) ss += __shfl_xor_sync(~0u, ss, m);
            if (nw) {
                const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * r * __ldg(nw + d + i);
            }
            const bool turn = !is_v && d < a.rot;
            if (a.interleaved) {
                if (turn) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 r = cs[d / 2 + i];
                        const float p = x[2 * i], n = x[2 * i + 1];
                        x[2 * i] = p * r.x - n * r.y;
                        x[2 * i + 1] = n * r.x + p * r.y;
                    }
                }
            } else if (a.rot) {
                const int half = a.rot / 2;
                const bool upper = d >= half;
                const int src = (tid & 31) + (d < a.rot ? (upper ? -half / 8 : half / 8) : 0);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = __shfl_sync(~0u, x[i], src);
                    if (turn) {
                        const float2 r = cs[(upper ? d - half : d) + i];
                        x[i] = upper ? x[i] * r.x + y * r.y : x[i] * r.x - y * r.y;
                    }
                }
            }
            if (c >= nch) continue;
            if (is_q || !E4M3) {
                const uint4 o = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                           pack_bf16x2(x[6], x[7]));
                void* p = is_q ? static_cast<void*>(a.q_out + t * a.out_stride + head * D + d)
                          : is_v ? a.v_cache + place + (head - a.Hq - a.Hk) * a.head_b + d * 2
                                 : a.k_cache + place + (head - a.Hq) * a.head_b + d * 2;
                *static_cast<uint4*>(p) = o;
            } else {
                const int h = is_v ? head - a.Hq - a.Hk : head - a.Hq;
                const float* sc = is_v ? a.v_scale : a.k_scale;
                if (sc) {
                    const float s = __ldg(sc + h);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], s);
                }
                *reinterpret_cast<uint2*>((is_v ? a.v_cache : a.k_cache) + place + h * a.head_b + d) = pack_e4m3x8(x);
            }
        }
    }
}
