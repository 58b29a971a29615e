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

__device__ __forceinline__ void set_status(int* status, int code) { atomicCAS(status, 0, code); }

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
        for (int i = 0; i < 4; ++i) out[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
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
    int32_t n, layer;
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

// One team of TEAM threads quantises what one call puts into one page, for one
// head of k or of v: the largest magnitude first, then the codes (the second
// read hits L1 or L2). Rows that the page held before are moved to the new
// scale if it is larger. TEAM = 32 for calls of a few tokens a sequence (decoding:
// one 128- or 256-byte row), 256 for prompts.
//
// Bound by HBM for prompts (2 bytes read, 1 written for each element), by
// latency for single tokens.
template <int TEAM, bool INT8>
__global__ void __launch_bounds__(256) cache_write_kernel(const __grid_constant__ CacheWriteParams p) {
    __shared__ uint32_t s_max[8];
    constexpr int kTeams = 256 / TEAM;
    const int lane = threadIdx.x % TEAM;
    const KvCache& c = p.c;
    // unit = (item, head, k or v), a team's own: the exits below are uniform over it
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kTeams + threadIdx.x / TEAM;
    const int per_item = 2 * c.heads;
    const int64_t item = unit / per_item;
    if (item >= p.items) return;
    const int sub = static_cast<int>(unit - item * per_item);
    const bool is_v = sub >= c.heads;
    const int head = is_v ? sub - c.heads : sub;

    const int i = p.cu == nullptr ? static_cast<int>(item) : item_sequence(p.cu, p.n, c.page_shift, item);
    const int64_t t0 = p.cu == nullptr ? item : __ldg(p.cu + i), t1 = p.cu == nullptr ? item + 1 : __ldg(p.cu + i + 1);
    const int seq = __ldg(p.seqs + i);
    const int64_t start = __ldg(p.starts + i);
    if (t0 < 0 || t1 < t0 || t1 > p.T) {
        if (lane == 0) set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);
        return;
    }
    if (seq == -1 || start == -1 || t0 == t1) return;
    if (seq < 0 || seq >= c.max_seqs || start < 0 || start + (t1 - t0) > __ldg(c.seq_lens + seq) ||
        start + (t1 - t0) > seq_capacity(c)) {
        if (lane == 0) set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
        return;
    }
    const int64_t which = p.cu == nullptr ? 0 : item - ((t0 >> c.page_shift) + 2 * static_cast<int64_t>(i));
    const int64_t slot = (start >> c.page_shift) + which;
    const int64_t lo = max(start, slot << c.page_shift), hi = min(start + (t1 - t0), (slot + 1) << c.page_shift);
    if (which < 0 || lo >= hi) return;
    const int page = __ldg(c.page_table + static_cast<int64_t>(seq) * c.max_pages + slot);
    if (page < 0 || page >= c.pages) {
        if (lane == 0) set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
        return;
    }
    if (__ldg(c.ref_counts + page) != 1) {  // a page that others read, or a free one
        if (lane == 0) set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);
        return;
    }
    const int row0 = static_cast<int>(lo & (c.page - 1)), rows = static_cast<int>(hi - lo);
    const __nv_bfloat16* src = is_v ? p.v + (t0 + lo - start) * p.vt + head * p.vh : p.k + (t0 + lo - start) * p.kt + head * p.kh;
    const int64_t src_row = is_v ? p.vt : p.kt;
    const int64_t place = static_cast<int64_t>(p.layer) * c.pages + page;
    uint8_t* dst = (is_v ? c.v : c.k) + place * page_elems(c) + static_cast<int64_t>(head) * c.page * c.dim;
    float* scale = (is_v ? c.v_scale : c.k_scale) + place * c.heads + head;
    const float held = row0 > 0 ? *scale : 0.f;

    const int vecs = c.dim / 8, shift = c.dim == 128 ? 4 : 3;  // 16-byte vectors of a row
    uint32_t most = 0;
    bool nan = false;
#pragma unroll 4
    for (int x = lane; x < rows * vecs; x += TEAM) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + (x >> shift) * src_row + (x & (vecs - 1)) * 8);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = ws[j] & 0x7FFFu, b = ws[j] >> 16 & 0x7FFFu;
            most = max(most, max(a < 0x7F80u ? a : 0u, b < 0x7F80u ? b : 0u));  // finite values only
            nan = nan || a > 0x7F80u || b > 0x7F80u;
        }
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (TEAM > 32) {
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) most = max(most, s_max[w]);
    }
    if (INT8 && nan) set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);  // (int8 has no NaN: stored as 0)
    __syncwarp();  // every lane has read the held scale
    const int e = scale_exp(most, INT8);
    const float fresh = exp2i(e);
    const float used = fmaxf(fresh, held);
    const float inv = used == fresh ? exp2i(-e) : __fdiv_rn(1.f, used);
    if (row0 > 0 && used != held) {
        const float ratio = __fdiv_rn(held, used);
        for (int x = lane; x < row0 * c.dim / 4; x += TEAM) {
            uint32_t* w = reinterpret_cast<uint32_t*>(dst) + x;
            float f[4];
            decode4<INT8>(*w, f);
            *w = encode4<INT8>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
        }
    }
    dst += static_cast<int64_t>(row0) * c.dim;
#pragma unroll 4
    for (int x = lane; x < rows * vecs; x += TEAM) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + (x >> shift) * src_row + (x & (vecs - 1)) * 8);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(ws[j] << 16) * inv;
            f[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u) * inv;
        }
        *reinterpret_cast<uint2*>(dst + x * 8) =
            make_uint2(encode4<INT8>(f[0], f[1], f[2], f[3]), encode4<INT8>(f[4], f[5], f[6], f[7]));
    }
    if (lane == 0) *scale = used;
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
    int32_t n, layer;
    int* status;
};

constexpr int kGatherTokens = 16;

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
// starts[i] + t - cu[i]. A block finds the places of kGatherTokens tokens, then
// streams their rows. Bound by HBM: 1 byte read, 2 written for each element.
template <bool INT8>
__global__ void __launch_bounds__(256) cache_gather_kernel(const __grid_constant__ CacheGatherParams p) {
    __shared__ int s_page[kGatherTokens], s_row[kGatherTokens];
    const KvCache& c = p.c;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kGatherTokens;
    if (threadIdx.x < kGatherTokens && first + threadIdx.x < p.T) {
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
    const int tokens = static_cast<int>(min(static_cast<int64_t>(kGatherTokens), p.T - first));
    const int shift = c.dim == 128 ? 4 : 3, vecs = c.dim / 8;
    const int per_token = c.heads * vecs;
    const int total = tokens * per_token;
    for (int which = 0; which < 2; ++which) {
        const uint8_t* codes = which ? p.c.v : p.c.k;
        const float* scales = which ? c.v_scale : c.k_scale;
        __nv_bfloat16* out = (which ? p.v : p.k) + first * per_token * 8;
#pragma unroll 4
        for (int x = threadIdx.x; x < total; x += 256) {
            const int t = x / per_token, hv = x - t * per_token;
            const int head = hv >> shift, vec = hv & (vecs - 1);
            uint4 r = make_uint4(0, 0, 0, 0);
            if (s_page[t] >= 0) {
                const int64_t place = static_cast<int64_t>(p.layer) * c.pages + s_page[t];
                const uint2 w = *reinterpret_cast<const uint2*>(
                    codes + ((place * c.heads + head) * c.page + s_row[t]) * c.dim + vec * 8);
                r = dequantise8<INT8>(w, __ldg(scales + place * c.heads + head));
            }
            *reinterpret_cast<uint4*>(out + static_cast<int64_t>(x) * 8) = r;
        }
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
        for (int r = threadIdx.x; r < total; r += kPlanThreads) {
            int lo = 0, hi = kPlanThreads - 1;  // the last sequence whose pages begin at or before r
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_off[mid] <= r)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int page = p.list[before + r];
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

// Copies `units` spans of 16 bytes with the block's share of the grid's threads.
template <typename F>
__device__ __forceinline__ void copy_vectors(int64_t begin, int64_t end, F place) {
    constexpr int kDeep = 8;  // 16-byte loads a thread has in flight
    for (int64_t x0 = begin + threadIdx.x; x0 < end; x0 += static_cast<int64_t>(blockDim.x) * kDeep) {
        uint4 v[kDeep];
        const uint4* from;
        uint4* to[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int64_t x = x0 + static_cast<int64_t>(j) * blockDim.x;
            if (x < end) {
                place(x, from, to[j]);
                v[j] = *from;
            }
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
            if (x0 + static_cast<int64_t>(j) * blockDim.x < end) *to[j] = v[j];
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
    // vectors: (layer, k or v, head, the page's first `rows` rows)
    const int64_t per_head = static_cast<int64_t>(rows) * c.dim / 16;
    const int64_t spans = static_cast<int64_t>(c.layers) * 2 * c.heads;
    const int64_t head_bytes = static_cast<int64_t>(c.page) * c.dim;
    const int64_t all = spans * per_head, share = (all + p.blocks - 1) / p.blocks;
    const int64_t begin = part * share;
    copy_vectors(begin, min(all, begin + share), [&](int64_t x, const uint4*& a, uint4*& b) {
        const int64_t span = x / per_head;
        const int64_t lk = span / c.heads, head = span - lk * c.heads;
        uint8_t* pool = (lk & 1) ? c.v : c.k;
        const int64_t base = (lk >> 1) * c.pages, in = (x - span * per_head) * 16;
        a = reinterpret_cast<const uint4*>(pool + ((base + old) * c.heads + head) * head_bytes + in);
        b = reinterpret_cast<uint4*>(pool + ((base + page) * c.heads + head) * head_bytes + in);
    });
    for (int64_t x = part * 256 + threadIdx.x; x < spans; x += p.blocks * 256) {
        const int64_t lk = x / c.heads, head = x - lk * c.heads;
        float* scale = (lk & 1) ? c.v_scale : c.k_scale;
        scale[((lk >> 1) * c.pages + page) * c.heads + head] = scale[((lk >> 1) * c.pages + old) * c.heads + head];
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

constexpr int kCompactChunk = 16384;  // bytes a block copies at a time

// Moves the pages (bound by HBM: each byte read once and written once) and
// renames them in the table.
__global__ void __launch_bounds__(256) cache_compact_kernel(const __grid_constant__ CacheCompactParams p) {
    const KvCache& c = p.c;
    const int live = p.header[0], movers = p.header[1];
    if (movers == 0) return;
    for (int seq = blockIdx.x; seq < c.max_seqs; seq += gridDim.x) {
        const int64_t len = c.seq_lens[seq];
        if (len < 0 || len > seq_capacity(c)) {
            if (threadIdx.x == 0) set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
            continue;
        }
        const int held = static_cast<int>((len + c.page - 1) >> c.page_shift);
        for (int x = threadIdx.x; x < held; x += 256) {
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
    const int64_t bytes = page_elems(c);
    const int64_t chunks = (bytes + kCompactChunk - 1) / kCompactChunk;
    const int64_t spans = static_cast<int64_t>(c.layers) * 2;
    const int64_t units = movers * spans * chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t chunk = u % chunks, ls = u / chunks;
        const int64_t lk = ls % spans;
        const int r = static_cast<int>(ls / spans);
        const int from = p.movers[r], to = p.holes[r];
        const int64_t base = (lk >> 1) * c.pages;
        uint8_t* pool = (lk & 1) ? c.v : c.k;
        const uint4* a = reinterpret_cast<const uint4*>(pool + (base + from) * bytes);
        uint4* b = reinterpret_cast<uint4*>(pool + (base + to) * bytes);
        const int64_t begin = chunk * kCompactChunk / 16, end = min(bytes, (chunk + 1) * kCompactChunk) / 16;
        copy_vectors(begin, end, [&](int64_t x, const uint4*& f, uint4*& t) {
            f = a + x;
            t = b + x;
        });
        if (chunk == 0) {
            float* scale = (lk & 1) ? c.v_scale : c.k_scale;
            for (int h = threadIdx.x; h < c.heads; h += 256)
                scale[(base + to) * c.heads + h] = scale[(base + from) * c.heads + h];
        }
    }
}

}  // namespace bsmt
