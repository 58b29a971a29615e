// The 8-bit paged cache: quantised writes, dequantised reads, and its pages
// (extend, fork, free, compact).
//
// Codes are e4m3 or int8, in pages of P tokens [layers, pages, Hkv, P, D], with
// one scale 2^e for each page and head of k and of v: the smallest power of two
// with amax <= top * 2^e, top = 448 or 127. Powers of two keep every step but
// the rounding to a code exact: x / 2^e, code * 2^e, and the move of held codes
// to a larger scale when later tokens of the page need one.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "async_copy.cuh"
#include "bsmt_serving.h"

namespace bsmt {

struct KvCache {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    int32_t* page_table;
    int32_t* seq_lens;
    int32_t* ref_counts;
    int32_t layers, pages, heads, page, page_shift, dim, max_seqs, max_pages, int8;
};

// N elements that are loaded or stored at once.
template <typename E, int N>
struct alignas(sizeof(E) * N) Pack {
    E v[N];
};

constexpr int kMinScaleExp = -120;  // a page of zeros has this scale

__device__ __forceinline__ int64_t page_elems(const KvCache& c) {
    return static_cast<int64_t>(c.heads) * c.page * c.dim;
}

// Tokens a sequence's table row can hold.
__device__ __forceinline__ int64_t seq_capacity(const KvCache& c) {
    return static_cast<int64_t>(c.max_pages) << c.page_shift;
}

// e of the smallest 2^e with amax <= top * 2^e, amax given as the bits of a
// non-negative finite bf16 (448 = 1.75 * 2^8, 127 = 1.984375 * 2^6).
__device__ __forceinline__ int scale_exp(uint32_t bits, bool int8) {
    const int x = static_cast<int>(bits >> 7) - 127;
    const int m = static_cast<int>(bits & 0x7Fu);
    const int e = int8 ? (x - 6 + (m > 0x7E)) : (x - 8 + (m > 0x60));
    return max(e, kMinScaleExp);  // (zero and subnormal amax: x = -127)
}

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// Two floats -> two e4m3 codes, round to nearest even, saturating (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (the low 16 bits) -> two halves, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return r;
}

__device__ __forceinline__ float2 half2_floats(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// float -> int8 code: nearest even, saturating; NaN gives 0.
__device__ __forceinline__ uint32_t int8_code(float x) {
    const int r = __float2int_rn(fminf(fmaxf(x, -127.f), 127.f));
    return static_cast<uint32_t>(x == x ? r : 0) & 0xFFu;
}

template <bool INT8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if (INT8) return int8_code(a) | int8_code(b) << 8 | int8_code(c) << 16 | int8_code(d) << 24;
    return e4m3x2(a, b) | e4m3x2(c, d) << 16;
}

template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t w, float out[4]) {
    if (INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)  // the float 2^23 + (code + 128), less 2^23 + 128
            out[i] = __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4B000000u, 0x7440 + i)) - 8388736.f;
    } else {
        const float2 a = half2_floats(e4m3x2_to_half2(w)), b = half2_floats(e4m3x2_to_half2(w >> 16));
        out[0] = a.x, out[1] = a.y, out[2] = b.x, out[3] = b.y;
    }
}

// ------------------------------------------------------------------ write
struct CacheWriteParams {
    KvCache c;
    const int32_t* seqs;
    const int32_t* starts;
    const int32_t* cu;  // NULL: one token a sequence
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    int64_t kt, kh, vt, vh;  // element strides: token, head
    int64_t T, items;
    int32_t n, layer, share;  // share: heads of k and v that one block of a prompt takes
    int* status;
};

// Largest i in [0, n) with base(i) = cu[i] / P + 2 i at most x. A sequence whose
// tokens touch m pages has m <= base(i + 1) - base(i) places, so the items of
// a ragged batch are found without a plan. (Not increasing cu: some i, in range.)
__device__ __forceinline__ int item_sequence(const int32_t* cu, int n, int shift, int64_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((static_cast<int64_t>(__ldg(cu + mid)) >> shift) + 2 * static_cast<int64_t>(mid) <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Where the tokens of one item go.
struct CacheItem {
    int64_t token;  // the first, in the call's pack
    int64_t place;  // layer * pages + page
    int row0, rows;
};

// False: nothing to write (an entry passed over, or one that is refused).
__device__ __forceinline__ bool cache_item(const CacheWriteParams& p, int64_t item, bool report, CacheItem& out) {
    const KvCache& c = p.c;
    const int i = p.cu == nullptr ? static_cast<int>(item) : item_sequence(p.cu, p.n, c.page_shift, item);
    const int64_t t0 = p.cu == nullptr ? item : __ldg(p.cu + i), t1 = p.cu == nullptr ? item + 1 : __ldg(p.cu + i + 1);
    const int seq = __ldg(p.seqs + i);
    const int64_t start = __ldg(p.starts + i);
    if (i == 0 && t0 != 0 && p.cu != nullptr && report) set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);  // (offsets begin at 0)
    if (t0 < 0 || t1 < t0 || t1 > p.T) {
        if (report) set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);
        return false;
    }
    if (seq == -1 || start == -1 || t0 == t1) return false;
    if (seq < 0 || seq >= c.max_seqs || start < 0 || start + (t1 - t0) > __ldg(c.seq_lens + seq) ||
        start + (t1 - t0) > seq_capacity(c)) {
        if (report) set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
        return false;
    }
    const int64_t which = p.cu == nullptr ? 0 : item - ((t0 >> c.page_shift) + 2 * static_cast<int64_t>(i));
    const int64_t slot = (start >> c.page_shift) + which;
    const int64_t lo = max(start, slot << c.page_shift), hi = min(start + (t1 - t0), (slot + 1) << c.page_shift);
    if (which < 0 || lo >= hi) return false;
    const int page = __ldg(c.page_table + static_cast<int64_t>(seq) * c.max_pages + slot);
    if (page < 0 || page >= c.pages) {
        if (report) set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
        return false;
    }
    if (__ldg(c.ref_counts + page) != 1) {  // a page that others read, or a free one
        if (report) set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);
        return false;
    }
    out.token = t0 + lo - start;
    out.place = static_cast<int64_t>(p.layer) * c.pages + page;
    out.row0 = static_cast<int>(lo & (c.page - 1));
    out.rows = static_cast<int>(hi - lo);
    return true;
}

// The largest magnitudes of a vector's even and odd values, as bf16 bits in two halves.
__device__ __forceinline__ uint32_t most_of(const uint4& w, uint32_t most) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = ws[j] & 0x7FFF7FFFu;
        asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(a));
    }
    return most;
}

// The same without infinities and NaN; notes whether there is a NaN.
__device__ __forceinline__ uint32_t most_finite(const uint4& w, uint32_t most, bool& nan) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = ws[j] & 0x7FFFu, b = ws[j] >> 16 & 0x7FFFu;
        nan = nan || a > 0x7F80u || b > 0x7F80u;
        const uint32_t f = (a < 0x7F80u ? a : 0u) | (b < 0x7F80u ? b : 0u) << 16;
        asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(f));
    }
    return most;
}

// Eight values times inv as codes. `plain`: all finite, within the codes' range.
template <bool INT8>
__device__ __forceinline__ uint2 encode8(const uint4& w, float inv, bool plain) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(ws[j] << 16);
        f[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
    }
    if (INT8 && plain) {
        // x * inv + 1.5 * 2^23 rounds to the nearest whole number, ties to even, into the low bits (x * inv is exact)
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(fmaf(f[j], inv, 12582912.f));
        return make_uint2(__byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410),
                          __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= inv;
    return make_uint2(encode4<INT8>(f[0], f[1], f[2], f[3]), encode4<INT8>(f[4], f[5], f[6], f[7]));
}

// The scale of a page's head once `most` is among its values, its inverse, and,
// where the page holds rows already and the scale grows, those rows under it.
template <bool INT8>
__device__ __forceinline__ float page_scale(uint32_t most, float held, int row0, uint8_t* codes, int dim, int lane, int team,
                                            float* inv) {
    const int e = scale_exp(most, INT8);
    const float fresh = exp2i(e);
    const float used = fmaxf(fresh, held);
    *inv = used == fresh ? exp2i(-e) : __fdiv_rn(1.f, used);
    if (row0 > 0 && used != held) {
        const float ratio = __fdiv_rn(held, used);
        for (int x = lane; x < row0 * dim / 4; x += team) {
            uint32_t* w = reinterpret_cast<uint32_t*>(codes) + x;
            float f[4];
            decode4<INT8>(*w, f);
            *w = encode4<INT8>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
        }
    }
    return used;
}

// A few tokens a sequence (decoding): a warp quantises what the call puts into one
// page, for one head of k or of v (one 128- or 256-byte row for one token). The
// largest magnitude first, then the codes; a second read of more rows than the
// first loop keeps hits L1. Bound by the latency of the chain from the list to the page.
template <bool INT8>
__global__ void __launch_bounds__(256) cache_write_rows_kernel(const __grid_constant__ CacheWriteParams p) {
    const int lane = threadIdx.x & 31;
    const KvCache& c = p.c;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);  // (item, k or v, head)
    const int per_item = 2 * c.heads;
    const int64_t item = unit / per_item;
    CacheItem it;
    if (item >= p.items || !cache_item(p, item, lane == 0, it)) return;
    const int sub = static_cast<int>(unit - item * per_item);
    const bool is_v = sub >= c.heads;
    const int head = is_v ? sub - c.heads : sub;
    const int64_t src_row = is_v ? p.vt : p.kt;
    const __nv_bfloat16* src = (is_v ? p.v + head * p.vh : p.k + head * p.kh) + it.token * src_row;
    uint8_t* dst = (is_v ? c.v : c.k) + it.place * page_elems(c) + static_cast<int64_t>(head) * c.page * c.dim;
    float* scale = (is_v ? c.v_scale : c.k_scale) + it.place * c.heads + head;
    const float held = it.row0 > 0 ? *scale : 0.f;
    const int vecs = c.dim / 8, shift = c.dim == 128 ? 4 : 3;  // 16-byte vectors of a row
    uint32_t both = 0;
    bool nan = false;
    for (int x = lane; x < it.rows * vecs; x += 32)
        both = most_finite(*reinterpret_cast<const uint4*>(src + (x >> shift) * src_row + (x & (vecs - 1)) * 8), both, nan);
    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(both & 0xFFFFu, both >> 16));
    if (INT8 && nan) set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);  // (int8 has no NaN: stored as 0)
    __syncwarp();  // every lane has read the held scale
    float inv;
    const float used = page_scale<INT8>(most, held, it.row0, dst, c.dim, lane, 32, &inv);
    dst += static_cast<int64_t>(it.row0) * c.dim;
    for (int x = lane; x < it.rows * vecs; x += 32)
        *reinterpret_cast<uint2*>(dst + x * 8) =
            encode8<INT8>(*reinterpret_cast<const uint4*>(src + (x >> shift) * src_row + (x & (vecs - 1)) * 8), inv, false);
    if (lane == 0) *scale = used;
}

// Prompts: a block quantises what the call puts into one page, for `share` of the
// 2 * Hkv heads of k and v, one after another. It finds the page once, holds a head's
// values in registers (NV vectors of 8 a thread: a page is NV * 2048 values at most)
// from the search for the largest to the codes, and has the next head's on their way
// meanwhile. Bound by HBM: 2 bytes read, 1 written for each element: 47k tokens of 8
// heads of 128 in 64 us (4.5 TB/s; 69 us with the three blocks an SM that 80 registers leave).
template <int NV, bool INT8>
__global__ void __launch_bounds__(256, NV <= 4 ? 4 : 2) cache_write_pages_kernel(const __grid_constant__ CacheWriteParams p) {
    __shared__ __align__(16) uint32_t s_most[2][8];
    const KvCache& c = p.c;
    const int groups = (2 * c.heads + p.share - 1) / p.share;
    const int64_t item = blockIdx.x / groups;
    CacheItem it;
    if (!cache_item(p, item, threadIdx.x == 0, it)) return;
    const int u0 = static_cast<int>(blockIdx.x - item * groups) * p.share, u1 = min(2 * c.heads, u0 + p.share);
    // the thread's vectors: one column of 8 values, every `step`th row
    const int shift = c.dim == 128 ? 4 : 3, row = threadIdx.x >> shift, step = 256 >> shift;
    const int col = (threadIdx.x & ((1 << shift) - 1)) * 8;
    const __nv_bfloat16* const k0 = p.k + (it.token + row) * p.kt + col;
    const __nv_bfloat16* const v0 = p.v + (it.token + row) * p.vt + col - static_cast<int64_t>(c.heads) * p.vh;
    const int64_t k_step = step * p.kt, v_step = step * p.vt;
    const int64_t head_bytes = static_cast<int64_t>(c.page) * c.dim, at = it.place * c.heads;  // of the page's first head
    auto load = [&](int u, uint4 w[NV]) {
        const bool is_v = u >= c.heads;
        const __nv_bfloat16* src = is_v ? v0 + u * p.vh : k0 + u * p.kh;
        const int64_t next_row = is_v ? v_step : k_step;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            w[j] = row + j * step < it.rows ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
            src += next_row;
        }
    };
    uint4 now[NV], next[NV];
    load(u0, now);
    for (int u = u0; u < u1; ++u) {
        const bool is_v = u >= c.heads;
        const int64_t place = at + (is_v ? u - c.heads : u);
        float* scale = (is_v ? c.v_scale : c.k_scale) + place;
        uint8_t* codes = (is_v ? c.v : c.k) + place * head_bytes;
        const float held = it.row0 > 0 ? *scale : 0.f;
        if (u + 1 < u1) load(u + 1, next);
        uint32_t both = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) both = most_of(now[j], both);
        const bool plain = (both & 0xFFFFu) < 0x7F80u && both < 0x7F800000u;
        if (!plain) {  // infinities or NaN among this thread's values
            bool nan = false;
            both = 0;
#pragma unroll
            for (int j = 0; j < NV; ++j) both = most_finite(now[j], both, nan);
            if (INT8 && nan) set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);  // (int8 has no NaN: stored as 0)
        }
        uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(both & 0xFFFFu, both >> 16));
        if ((threadIdx.x & 31) == 0) s_most[u & 1][threadIdx.x >> 5] = most;
        __syncthreads();
        const uint4 m0 = *reinterpret_cast<const uint4*>(s_most[u & 1]), m1 = *reinterpret_cast<const uint4*>(s_most[u & 1] + 4);
        most = max(max(max(m0.x, m0.y), max(m0.z, m0.w)), max(max(m1.x, m1.y), max(m1.z, m1.w)));
        float inv;
        const float used = page_scale<INT8>(most, held, it.row0, codes, c.dim, threadIdx.x, 256, &inv);
        uint8_t* dst = codes + it.row0 * c.dim + threadIdx.x * 8;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (row + j * step < it.rows) *reinterpret_cast<uint2*>(dst + j * 2048) = encode8<INT8>(now[j], inv, plain);
        if (threadIdx.x == 0) *scale = used;
#pragma unroll
        for (int j = 0; j < NV; ++j) now[j] = next[j];
    }
}

// ----------------------------------------------------------------- gather
struct CacheGatherParams {
    KvCache c;
    const int32_t* seqs;
    const int32_t* starts;  // NULL: 0
    const int32_t* cu;      // NULL: one token a sequence
    __nv_bfloat16* k;
    __nv_bfloat16* v;
    int64_t T;
    int32_t n, layer, tokens;  // tokens of one block
    int* status;
};

constexpr int kGatherTokens = 8;  // at most

// code * 2^e in bf16 (exact while the value is in bf16's normal range: a code
// has at most 8 significant bits).
template <bool INT8>
__device__ __forceinline__ uint4 dequantise8(uint2 w, float scale) {
    float f[8];
    decode4<INT8>(w.x, f);
    decode4<INT8>(w.y, f + 4);
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j] * scale, f[2 * j + 1] * scale);
        r[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// k, v [T, Hkv, D] of tokens of the cache: token t of sequence i is position
// starts[i] + t - cu[i]. A block finds the places of its tokens, then streams
// their rows. Bound by HBM: 1 byte read, 2 written for each element: 47k tokens of 8
// heads of 128 in 53 us (5.5 TB/s; 59 us with 32 tokens a block, 57 with 4).
template <bool INT8>
__global__ void __launch_bounds__(256) cache_gather_kernel(const __grid_constant__ CacheGatherParams p) {
    __shared__ int s_page[kGatherTokens], s_row[kGatherTokens];
    const KvCache& c = p.c;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tokens;
    if (threadIdx.x < p.tokens && first + threadIdx.x < p.T) {
        const int64_t t = first + threadIdx.x;
        int i = static_cast<int>(t);
        int64_t begin = t;
        bool there = true, bad = false;
        if (p.cu != nullptr) {
            int lo = 0, hi = p.n;  // largest i with cu[i] <= t; n: behind the last sequence
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (__ldg(p.cu + mid) <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            i = lo;
            begin = __ldg(p.cu + i);
            there = i < p.n;
            bad = begin < 0 || begin > t;
        }
        int page = -1, row = 0;
        if (bad) {
            set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);
        } else if (there) {
            const int seq = __ldg(p.seqs + i);
            const int start = p.starts == nullptr ? 0 : __ldg(p.starts + i);
            if (seq != -1 && start != -1) {
                const int64_t pos = start + (t - begin);
                if (seq < 0 || seq >= c.max_seqs || start < 0 || pos >= __ldg(c.seq_lens + seq) || pos >= seq_capacity(c)) {
                    set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
                } else {
                    page = __ldg(c.page_table + static_cast<int64_t>(seq) * c.max_pages + (pos >> c.page_shift));
                    row = static_cast<int>(pos & (c.page - 1));
                    if (page < 0 || page >= c.pages) {
                        set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
                        page = -1;
                    }
                }
            }
        }
        s_page[threadIdx.x] = page;
        s_row[threadIdx.x] = row;
    }
    __syncthreads();
    // 16 codes at a time, of k's rows and then of v's
    const int tokens = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.T - first));
    const int shift = c.dim == 128 ? 3 : 2, per_token = c.heads << shift;
    const int half = tokens * per_token;
#pragma unroll 4
    for (int x = threadIdx.x; x < 2 * half; x += 256) {
        const bool is_v = x >= half;
        const int y = is_v ? x - half : x;
        const int t = static_cast<uint32_t>(y) / static_cast<uint32_t>(per_token), hv = y - t * per_token;
        const int head = hv >> shift, vec = hv & ((1 << shift) - 1);
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
        if (s_page[t] >= 0) {
            const int64_t place = (static_cast<int64_t>(p.layer) * c.pages + s_page[t]) * c.heads + head;
            const uint4 w = __ldg(reinterpret_cast<const uint4*>((is_v ? c.v : c.k) + (place * c.page + s_row[t]) * c.dim + vec * 16));
            const float scale = __ldg((is_v ? c.v_scale : c.k_scale) + place);
            lo = dequantise8<INT8>(make_uint2(w.x, w.y), scale);
            hi = dequantise8<INT8>(make_uint2(w.z, w.w), scale);
        }
        uint4* out = reinterpret_cast<uint4*>((is_v ? p.v : p.k) + (first * per_token + y) * 16);
        out[0] = lo;
        out[1] = hi;
    }
}

// ------------------------------------------------------------------ pages
// Page bookkeeping runs in one block: its order is the list's order and the
// pages' order, so what it does is the same every time. Its refusals are
// all-or-nothing: nothing is written before every check has passed.
constexpr int kPlanThreads = 1024;

// Exclusive prefix sum over the block and the total (all threads call).
__device__ __forceinline__ int block_scan(int x, int* total, int* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += y;
    }
    __syncthreads();  // (s_warp may still be read from the call before)
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int before = 0, sum = 0;
    // every thread adds up the warps' totals (32 shared reads, broadcast)
    int w = s_warp[lane];
    int wi = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, wi, d);
        if (lane >= d) wi += y;
    }
    before = __shfl_sync(0xFFFFFFFFu, wi - w, warp);
    sum = __shfl_sync(0xFFFFFFFFu, wi, 31);
    *total = sum;
    return before + incl - x;
}

constexpr int kScanInts = 16;  // page counts of one thread in one step of a pool scan

// The step's 16 counts of this thread: which of them are free (bit i).
__device__ __forceinline__ uint32_t free_bits(const int32_t* refs, int pages, int64_t at, bool want_free) {
    uint32_t bits = 0;
    if (at + kScanInts <= pages) {
        int4 v[kScanInts / 4];
#pragma unroll
        for (int j = 0; j < kScanInts / 4; ++j) v[j] = *reinterpret_cast<const int4*>(refs + at + 4 * j);
#pragma unroll
        for (int j = 0; j < kScanInts / 4; ++j) {
            bits |= static_cast<uint32_t>(v[j].x <= 0) << (4 * j) | static_cast<uint32_t>(v[j].y <= 0) << (4 * j + 1) |
                    static_cast<uint32_t>(v[j].z <= 0) << (4 * j + 2) | static_cast<uint32_t>(v[j].w <= 0) << (4 * j + 3);
        }
        return want_free ? bits : ~bits & 0xFFFFu;
    }
    for (int j = 0; j < kScanInts; ++j)
        if (at + j < pages && (refs[at + j] <= 0) == want_free) bits |= 1u << j;
    return bits;
}

// Writes the lowest `want` free pages to list, ascending. Returns how many
// there are, at most `want` (all threads call; ends with a barrier).
__device__ __forceinline__ int find_free(const KvCache& c, int want, int32_t* list, int* s_warp) {
    int found = 0;
    for (int64_t at = 0; at < c.pages && found < want; at += kPlanThreads * kScanInts) {
        const int64_t mine = at + static_cast<int64_t>(threadIdx.x) * kScanInts;
        uint32_t bits = mine < c.pages ? free_bits(c.ref_counts, c.pages, mine, true) : 0u;
        int total;
        int rank = found + block_scan(__popc(bits), &total, s_warp);
        for (; bits != 0u && rank < want; bits &= bits - 1, ++rank)
            list[rank] = static_cast<int32_t>(mine) + __ffs(bits) - 1;
        found += total;
    }
    __syncthreads();
    return min(found, want);
}

// Marks seq in the bitmap; false if it was marked already.
__device__ __forceinline__ bool mark_once(uint32_t* bitmap, int seq) {
    const uint32_t bit = 1u << (seq & 31);
    return (atomicOr(bitmap + (seq >> 5), bit) & bit) == 0u;
}

struct CacheExtendParams {
    KvCache c;
    const int32_t* seqs;
    const int32_t* counts;  // NULL: 1 each
    int32_t* starts;
    int32_t* list;  // workspace [pages]
    int32_t n;
    int* status;
};

// Grows n sequences by counts[i] tokens: pages for them, their new lengths, and
// the old ones in starts. Latency bound (one block): the lengths are one
// dependent read each, the pool one pass over ref_counts up to the last page taken.
__global__ void __launch_bounds__(kPlanThreads) cache_extend_kernel(const __grid_constant__ CacheExtendParams p) {
    extern __shared__ uint32_t s_bitmap[];
    __shared__ int s_warp[32], s_bad, s_off[kPlanThreads], s_have[kPlanThreads], s_seq[kPlanThreads];
    __shared__ unsigned long long s_need;
    const KvCache& c = p.c;
    const int words = (c.max_seqs + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kPlanThreads) s_bitmap[i] = 0;
    if (threadIdx.x == 0) s_bad = 0, s_need = 0;
    __syncthreads();
    unsigned long long need = 0;
    int bad = 0;
    for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
        const int seq = p.seqs[i], count = p.counts == nullptr ? 1 : p.counts[i];
        if (seq == -1) continue;
        if (seq < 0 || seq >= c.max_seqs) {
            bad = BSMT_ERR_DEVICE_BOUNDS;
            continue;
        }
        const int64_t len = c.seq_lens[seq];
        if (!mark_once(s_bitmap, seq) || count < 0) {
            bad = BSMT_ERR_DEVICE_PRECONDITION;
        } else if (len < 0 || len > seq_capacity(c)) {
            bad = BSMT_ERR_DEVICE_BOUNDS;
        } else if (len + count > seq_capacity(c)) {
            bad = BSMT_ERR_DEVICE_CAPACITY;
        } else if (count > 0) {
            if (len & (c.page - 1)) {  // the page that the tokens go on in is this sequence's alone
                const int page = c.page_table[static_cast<int64_t>(seq) * c.max_pages + (len >> c.page_shift)];
                if (page < 0 || page >= c.pages)
                    bad = BSMT_ERR_DEVICE_BOUNDS;
                else if (c.ref_counts[page] != 1)
                    bad = BSMT_ERR_DEVICE_PRECONDITION;
            }
            need += ((len + count + c.page - 1) >> c.page_shift) - ((len + c.page - 1) >> c.page_shift);
        }
    }
    if (need != 0) atomicAdd(&s_need, need);
    if (bad != 0) atomicMax(&s_bad, bad);
    __syncthreads();
    bad = s_bad;
    const int64_t total_need = static_cast<int64_t>(s_need);
    if (bad == 0 && total_need > c.pages) bad = BSMT_ERR_DEVICE_CAPACITY;
    if (bad == 0 && total_need > 0 && find_free(c, static_cast<int>(total_need), p.list, s_warp) < total_need)
        bad = BSMT_ERR_DEVICE_CAPACITY;
    if (bad != 0) {
        for (int i = threadIdx.x; i < p.n; i += kPlanThreads) p.starts[i] = -1;
        if (threadIdx.x == 0) set_status(p.status, bad);
        return;
    }
    int before = 0;
    for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        int seq = -1, pages = 0, have = 0;
        if (i < p.n) {
            seq = p.seqs[i];
            int start = -1;
            if (seq >= 0) {
                const int count = p.counts == nullptr ? 1 : p.counts[i];
                start = c.seq_lens[seq];
                have = static_cast<int>((static_cast<int64_t>(start) + c.page - 1) >> c.page_shift);
                pages = static_cast<int>((static_cast<int64_t>(start) + count + c.page - 1) >> c.page_shift) - have;
                c.seq_lens[seq] = start + count;
            }
            p.starts[i] = start;
        }
        int total;
        s_off[threadIdx.x] = block_scan(pages, &total, s_warp);
        s_have[threadIdx.x] = have;
        s_seq[threadIdx.x] = seq;
        __syncthreads();
#pragma unroll 4
        for (int r = threadIdx.x; r < total; r += kPlanThreads) {
            const int page = __ldcg(p.list + before + r);
            int lo = 0, hi = kPlanThreads - 1;  // the last sequence whose pages begin at or before r
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_off[mid] <= r)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            c.page_table[static_cast<int64_t>(s_seq[lo]) * c.max_pages + s_have[lo] + r - s_off[lo]] = page;
            c.ref_counts[page] = 1;
        }
        before += total;
        __syncthreads();
    }
}

struct CacheForkParams {
    KvCache c;
    const int32_t* src;
    const int32_t* dst;
    int32_t* list;   // workspace [pages]
    int2* jobs;      // workspace [n]: the parent's length (-1: none), the copy of its last page (-1: none)
    int32_t n, blocks;  // blocks of one fork
    int* status;
};

// Checks a fork, hands out the pages of the parents' last, partial pages, and
// sets the children's lengths.
__global__ void __launch_bounds__(kPlanThreads) cache_fork_plan_kernel(const __grid_constant__ CacheForkParams p) {
    extern __shared__ uint32_t s_bitmap[];
    __shared__ int s_warp[32], s_bad, s_need;
    const KvCache& c = p.c;
    const int words = (c.max_seqs + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kPlanThreads) s_bitmap[i] = 0;
    if (threadIdx.x == 0) s_bad = 0, s_need = 0;
    __syncthreads();
    int bad = 0, need = 0;
    for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
        const int src = p.src[i], dst = p.dst[i];
        int len = -1;
        if (src != -1 && dst != -1) {
            if (src < 0 || src >= c.max_seqs || dst < 0 || dst >= c.max_seqs) {
                bad = BSMT_ERR_DEVICE_BOUNDS;
            } else {
                len = c.seq_lens[src];
                if (len < 0 || len > seq_capacity(c)) {
                    bad = BSMT_ERR_DEVICE_BOUNDS;
                } else if (!mark_once(s_bitmap, dst) || c.seq_lens[dst] != 0) {
                    bad = BSMT_ERR_DEVICE_PRECONDITION;
                } else if (len & (c.page - 1)) {
                    const int page = c.page_table[static_cast<int64_t>(src) * c.max_pages + (len >> c.page_shift)];
                    if (page < 0 || page >= c.pages) bad = BSMT_ERR_DEVICE_BOUNDS;
                    ++need;
                }
            }
        }
        p.jobs[i] = make_int2(len, -1);
    }
    if (need != 0) atomicAdd(&s_need, need);
    if (bad != 0) atomicMax(&s_bad, bad);
    __syncthreads();
    bad = s_bad;
    need = s_need;
    if (bad == 0 && need > c.pages) bad = BSMT_ERR_DEVICE_CAPACITY;
    if (bad == 0 && need > 0 && find_free(c, need, p.list, s_warp) < need) bad = BSMT_ERR_DEVICE_CAPACITY;
    if (bad != 0) {
        for (int i = threadIdx.x; i < p.n; i += kPlanThreads) p.jobs[i] = make_int2(-1, -1);
        if (threadIdx.x == 0) set_status(p.status, bad);
        return;
    }
    int before = 0;
    for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        const int len = i < p.n ? p.jobs[i].x : -1;
        const bool part = len > 0 && (len & (c.page - 1)) != 0;
        int total;
        const int rank = before + block_scan(part ? 1 : 0, &total, s_warp);
        if (len >= 0) {
            c.seq_lens[p.dst[i]] = len;
            if (part) {
                const int page = p.list[rank];
                c.ref_counts[page] = 1;
                p.jobs[i].y = page;
            }
        }
        before += total;
    }
}

// The children's table rows and the counts of the pages they share, and the
// copies of the partial pages: the rows that hold tokens, in every layer.
__global__ void __launch_bounds__(256) cache_fork_kernel(const __grid_constant__ CacheForkParams p) {
    const KvCache& c = p.c;
    const int i = blockIdx.x / p.blocks, part = blockIdx.x - i * p.blocks;
    const int2 job = p.jobs[i];
    const int len = job.x;
    if (len < 0) return;
    const int src = p.src[i], dst = p.dst[i];
    const int full = len >> c.page_shift, rows = len & (c.page - 1);
    const int32_t* from = c.page_table + static_cast<int64_t>(src) * c.max_pages;
    int32_t* to = c.page_table + static_cast<int64_t>(dst) * c.max_pages;
    for (int x = part * 256 + threadIdx.x; x < full; x += p.blocks * 256) {
        const int page = from[x];
        to[x] = page;
        if (page < 0 || page >= c.pages)
            set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
        else
            atomicAdd(c.ref_counts + page, 1);
    }
    if (rows == 0) return;
    const int old = from[full], page = job.y;
    if (part == 0 && threadIdx.x == 0) to[full] = page;
    // a warp for each (layer, k or v, head): the page's first `rows` rows
    const int spans = c.layers * 2 * c.heads, vectors = rows * c.dim / 16;
    const int64_t head_bytes = static_cast<int64_t>(c.page) * c.dim;
    for (int span = part * 8 + (threadIdx.x >> 5); span < spans; span += p.blocks * 8) {
        const int lk = span / c.heads, head = span - lk * c.heads;
        uint8_t* pool = (lk & 1) ? c.v : c.k;
        const int64_t base = static_cast<int64_t>(lk >> 1) * c.pages;
        const uint4* a = reinterpret_cast<const uint4*>(pool + ((base + old) * c.heads + head) * head_bytes);
        uint4* b = reinterpret_cast<uint4*>(pool + ((base + page) * c.heads + head) * head_bytes);
        constexpr int kDeep = 8;  // 16-byte loads a thread has in flight
        for (int x0 = threadIdx.x & 31; x0 < vectors; x0 += 32 * kDeep) {
            uint4 v[kDeep];
#pragma unroll
            for (int j = 0; j < kDeep; ++j)
                if (x0 + 32 * j < vectors) v[j] = a[x0 + 32 * j];
#pragma unroll
            for (int j = 0; j < kDeep; ++j)
                if (x0 + 32 * j < vectors) b[x0 + 32 * j] = v[j];
        }
    }
    for (int x = part * 256 + threadIdx.x; x < spans; x += p.blocks * 256) {
        const int lk = x / c.heads, head = x - lk * c.heads;
        float* scale = (lk & 1) ? c.v_scale : c.k_scale;
        const int64_t base = static_cast<int64_t>(lk >> 1) * c.pages;
        scale[(base + page) * c.heads + head] = scale[(base + old) * c.heads + head];
    }
}

// Empties sequences: one block each. A sequence listed twice is emptied once
// (its length is exchanged for 0 atomically).
__global__ void __launch_bounds__(256) cache_free_kernel(const __grid_constant__ KvCache c, const int32_t* seqs,
                                                         int* status) {
    __shared__ int s_len;
    const int seq = seqs[blockIdx.x];
    if (seq == -1) return;
    if (seq < 0 || seq >= c.max_seqs) {
        if (threadIdx.x == 0) set_status(status, BSMT_ERR_DEVICE_BOUNDS);
        return;
    }
    if (threadIdx.x == 0) s_len = atomicExch(c.seq_lens + seq, 0);
    __syncthreads();
    const int64_t len = s_len;
    if (len < 0 || len > seq_capacity(c)) {
        if (threadIdx.x == 0) set_status(status, BSMT_ERR_DEVICE_BOUNDS);
        return;
    }
    const int held = static_cast<int>((len + c.page - 1) >> c.page_shift);
    for (int x = threadIdx.x; x < held; x += blockDim.x) {
        int32_t* entry = c.page_table + static_cast<int64_t>(seq) * c.max_pages + x;
        const int page = *entry;
        *entry = -1;
        if (page < 0 || page >= c.pages) {
            set_status(status, BSMT_ERR_DEVICE_BOUNDS);
        } else if (atomicSub(c.ref_counts + page, 1) <= 0) {
            atomicAdd(c.ref_counts + page, 1);  // it was free: its count stays
            set_status(status, BSMT_ERR_DEVICE_PRECONDITION);
        }
    }
}

struct CacheCompactParams {
    KvCache c;
    int32_t* live;    // out [1]: pages in use
    int32_t* header;  // workspace [4]: pages in use, pages that move
    int32_t* holes;   // workspace [pages]
    int32_t* movers;  // workspace [pages]
    int32_t* to;      // workspace [pages]: where a page behind the first `live` goes, -1 for a free one
    int* status;
};

// The pages in use behind the first `live` places go, in order, to the free
// ones among those places. No page is both source and target. The counts move
// here, the pages and the table's names in the kernel that follows.
__global__ void __launch_bounds__(kPlanThreads) cache_compact_plan_kernel(const __grid_constant__ CacheCompactParams p) {
    __shared__ int s_warp[32];
    const KvCache& c = p.c;
    int mine_live = 0;
    for (int64_t at = static_cast<int64_t>(threadIdx.x) * kScanInts; at < c.pages; at += kPlanThreads * kScanInts)
        mine_live += __popc(free_bits(c.ref_counts, c.pages, at, false));
    int live;
    block_scan(mine_live, &live, s_warp);
    int holes = 0, movers = 0;
    for (int64_t at = 0; at < c.pages; at += kPlanThreads * kScanInts) {
        const int64_t mine = at + static_cast<int64_t>(threadIdx.x) * kScanInts;
        uint32_t hole = 0, mover = 0;
        if (mine < c.pages) {
            const uint32_t in_front = live <= mine ? 0u : live >= mine + kScanInts ? 0xFFFFu : (1u << (live - mine)) - 1u;
            const uint32_t unused = free_bits(c.ref_counts, c.pages, mine, true);
            hole = unused & in_front;
            mover = free_bits(c.ref_counts, c.pages, mine, false) & ~in_front;
            for (uint32_t none = unused & ~in_front; none != 0u; none &= none - 1)
                p.to[mine + __ffs(none) - 1] = -1;
        }
        int total;  // both counts in one scan: at most 16384 each
        const int both = block_scan(__popc(hole) | __popc(mover) << 16, &total, s_warp);
        int h = holes + (both & 0xFFFF), m = movers + (both >> 16);
        for (; hole != 0u; hole &= hole - 1) p.holes[h++] = static_cast<int32_t>(mine) + __ffs(hole) - 1;
        for (; mover != 0u; mover &= mover - 1) p.movers[m++] = static_cast<int32_t>(mine) + __ffs(mover) - 1;
        holes += total & 0xFFFF;
        movers += total >> 16;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < movers; r += kPlanThreads) {
        const int from = p.movers[r], to = p.holes[r];
        p.to[from] = to;
        c.ref_counts[to] = c.ref_counts[from];
        c.ref_counts[from] = 0;
    }
    if (threadIdx.x == 0) {
        p.header[0] = live;
        p.header[1] = movers;
        *p.live = live;
    }
}

constexpr int kCompactChunk = 16384;  // bytes of one copy
constexpr int kCompactSlots = 4;
constexpr int kCompactSmem = kCompactChunk * kCompactSlots;

// Moves the pages and renames them in the table. One thread of a block runs a ring
// of bulk copies, global to shared to global, four of 16 KB under way; the others
// rename and move the scales. Bound by HBM: each byte is read once and written once.
__global__ void __launch_bounds__(128) cache_compact_kernel(const __grid_constant__ CacheCompactParams p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t s_bars[kCompactSlots];
    const KvCache& c = p.c;
    const int live = p.header[0], movers = p.header[1];
    if (movers == 0) return;
    const int64_t spans = static_cast<int64_t>(c.layers) * 2;  // (layer, k or v)
    if (threadIdx.x == 0) {
        const uint32_t bars = shared_addr(s_bars), slots = shared_addr(ring);
        for (int i = 0; i < kCompactSlots; ++i) bar_init(bars + 8 * i);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        const int64_t bytes = page_elems(c);
        const int chunks = static_cast<int>((bytes + kCompactChunk - 1) / kCompactChunk);
        const int64_t units = movers * spans * chunks;
        auto find = [&](int64_t u, const uint8_t*& from, uint8_t*& to) -> uint32_t {
            const int64_t span = u / chunks;
            const int chunk = static_cast<int>(u - span * chunks);
            const int64_t r = span / spans, lk = span - r * spans;
            uint8_t* pool = ((lk & 1) ? c.v : c.k) + (lk >> 1) * c.pages * bytes + static_cast<int64_t>(chunk) * kCompactChunk;
            from = pool + p.movers[r] * bytes;
            to = pool + p.holes[r] * bytes;
            return static_cast<uint32_t>(min(static_cast<int64_t>(kCompactChunk), bytes - static_cast<int64_t>(chunk) * kCompactChunk));
        };
        // load unit n, then store unit n - (slots - 2) that came meanwhile
        constexpr int kLag = kCompactSlots - 2;
        uint8_t* to_q[kCompactSlots];
        uint32_t size_q[kCompactSlots];
        int64_t n = 0;
        for (int64_t u = blockIdx.x; ; u += gridDim.x, ++n) {
            const bool more = u < units;
            if (!more && u - static_cast<int64_t>(kLag) * gridDim.x >= units) break;
#pragma unroll
            for (int q = 0; q < kCompactSlots; ++q) {
                if (more && n % kCompactSlots == q) {
                    const uint8_t* from;
                    size_q[q] = find(u, from, to_q[q]);
                    bulk_wait_read<1>();  // the store from this slot, two stores ago, has left it
                    bar_expect(bars + 8 * q, size_q[q]);
                    bulk_load(slots + q * kCompactChunk, from, size_q[q], bars + 8 * q);
                }
            }
            const int64_t done = n - kLag;
            if (done < 0) continue;
#pragma unroll
            for (int q = 0; q < kCompactSlots; ++q) {
                if (done % kCompactSlots == q && u - static_cast<int64_t>(kLag) * gridDim.x < units) {
                    bar_wait(bars + 8 * q, static_cast<uint32_t>(done / kCompactSlots) & 1u, p.status);
                    bulk_store(to_q[q], slots + q * kCompactChunk, size_q[q]);
                }
            }
        }
        bulk_wait_all();
    } else if (threadIdx.x >= 32) {
        const int tid = threadIdx.x - 32;
        for (int seq = blockIdx.x; seq < c.max_seqs; seq += gridDim.x) {
            const int64_t len = c.seq_lens[seq];
            if (len < 0 || len > seq_capacity(c)) {
                if (tid == 0) set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
                continue;
            }
            const int held = static_cast<int>((len + c.page - 1) >> c.page_shift);
            for (int x = tid; x < held; x += 96) {
                int32_t* entry = c.page_table + static_cast<int64_t>(seq) * c.max_pages + x;
                const int page = *entry;
                if (page < 0 || page >= c.pages) {
                    set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
                } else if (page >= live) {
                    const int to = p.to[page];
                    if (to < 0)
                        set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);  // a free page in a table row: left as it is
                    else
                        *entry = to;
                }
            }
        }
        const int64_t scales = movers * spans * c.heads;
        for (int64_t x = static_cast<int64_t>(blockIdx.x) * 96 + tid; x < scales; x += static_cast<int64_t>(gridDim.x) * 96) {
            const int64_t span = x / c.heads, head = x - span * c.heads;
            const int64_t r = span / spans, lk = span - r * spans;
            float* scale = ((lk & 1) ? c.v_scale : c.k_scale) + (lk >> 1) * c.pages * c.heads + head;
            scale[static_cast<int64_t>(p.holes[r]) * c.heads] = scale[static_cast<int64_t>(p.movers[r]) * c.heads];
        }
    }
}

}  // namespace bsmt
