// Attention of the newest tokens of many sequences over the 8-bit paged cache.
//
//   out = softmax_j(mod(scale * q . k_j), masked) v,  k_j = code * k_scale[page, head]
//
// A unit is (sequence, row tile, kv head): a row is one query token with one
// query head of the kv head's group, a row tile 8 * NT of them. A unit's keys
// are cut into tiles of 32 tokens; tiles that no row sees are never read. All
// units' tiles form one list that is cut into equal shares, one for each block,
// so sequences of any lengths keep all blocks busy to the end. A unit that a
// share boundary cuts leaves parts (O, the running maxima and the sum, in fp32)
// in the workspace, which paged_combine_kernel joins in a fixed order.
//
// Bound by HBM: K and V codes are read once. Each warp of a block takes every
// fourth tile of the share and has its own ring of slots, which TMA fills: one copy
// of 4 KB for the K and one for the V of a tile (two of 2 KB with pages of 16), all
// four warps of three blocks an SM keeping some 150 KB loaded or on their way. The
// contraction's order is free, so a lane's 16 bytes of a K row are the four k
// positions of four MMA steps, and its 16 bytes of a V row are one row of each of 16
// half output tiles: wide shared loads, no transposes, no barrier between warps.
//
// The products are S^T = K q^T and O^T = V^T P^T: tokens and then columns of V are
// the 16 rows of mma.sync m16n8k16, the query rows its 8 columns. A decoded token
// has few rows, so this wastes less of the unit, and half the registers, of the
// other order. P^T goes from the first product's result to the second's operand
// by movmatrix. Codes become halves exactly (e4m3 by cvt, int8 by byte permutes);
// q, scaled by a power of two for each row, becomes halves exactly down to 2^-28
// of the row's largest value. tcgen05 takes 8-bit operands only in pairs, which would round q
// and P to 8 bits, and 16-bit ones from shared or tensor memory, which would cost
// a write of every converted tile; eight rows need no such rate.
//
// Softmax in base 2 with two references for each row: m of the scores, for the
// sum l, and mo of score + log2(v_scale), for O, so that P * v_scale, a half, stays
// in range whatever the pages' scales are. They follow the running maxima lazily, mo
// at a distance that lets P use a half's range to the top.
#pragma once
#include <cfloat>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "async_copy.cuh"
#include "kv_cache.cuh"
#include "mask_dnf.cuh"

namespace bsmt {

constexpr int kCombineWarps = 4;
constexpr int kTileTokens = 32;
constexpr float kLazy = 8.f;  // log2 by which a score may pass its reference
// log2 by which O's reference stays below the largest score + log2(v_scale): P * v_scale then lies below 2^(8 + 7), inside
// a half, and a half's smallest step, 2^-24, is 2^-31 of the largest term: many small terms beside one large one count.
constexpr float kRoom = 7.f;
constexpr float kRoomInv = 0x1p-7f;

struct PagedParams {
    KvCache c;
    const __nv_bfloat16* q;  // [T, Hq, D]
    const int32_t* seqs;
    const int32_t* cu;  // NULL: one token a sequence
    __nv_bfloat16* out;
    float* lse;       // [Hq, T]
    float* part_o;    // [2 * blocks][8 * NT][D]
    float* part_m;    // [2 * blocks][8 * NT][4]: m, mo, l
    int32_t* heads_of_parts;  // [blocks][8]: a cut unit that begins in this block
    const float* slopes;
    int64_t T;
    int32_t n, layer, Hq, group, min_share;
    float scale, cap;
    float cap_inv;  // 2 log2(e) / cap up to a cap of 64, beyond 1 / cap; at most the largest float
    int32_t alibi_first, alibi_h0, alibi_heads, softcap;
    int* status;
};

// Three blocks an SM with 16 KB of slots a warp; with NT = 4 (D = 64 alone) two with
// 24 KB. (NT = 2 at D = 128, 24 sequences up to 64k with 16 rows each, when it was chosen: 326 us
// in three blocks of 168 registers, 363 in two of 255; 317 us since. The three spill some: 20 to 204
// bytes of stores, by type and modifiers, the two none.) A slot holds the K or the V codes of a tile.
template <int D, int NT>
struct PagedShape {
    static constexpr int kBlocks = NT > 2 ? 2 : 3;  // of an SM
    static constexpr int kWarps = 4;
    static constexpr int kSlot = kTileTokens * D;
    static constexpr int kDeep = (kBlocks == 2 ? 3 : 2) * (128 / D);  // tiles a warp has loaded or on their way
    static constexpr int kWarpBytes = 2 * kDeep * kSlot;
    static constexpr int kPitch = D + 4;  // floats of a row where the warps' parts meet (in the slots)
    static_assert(8 * NT * (kPitch + 4) * 4 <= kWarpBytes, "a warp's part fits its slots");
    static constexpr int kQ = kWarps * kWarpBytes;
    static constexpr int kSmem = kQ + (NT > 1 ? NT * (D / 16) * 256 : 0) + 1024;  // NT > 1: q's fragments; alignment
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(u) = 1 - 2 / (exp(2 u) + 1), off by 2^-23 or so; for small u, where that would be much of the value, the
// first terms of its series (the next is below 2^-26 of it).
__device__ __forceinline__ float tanh_fast(float u) {
    const float q = u * u;
    const float series = u * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
    const float direct = 1.f - 2.f * rcp_fast(exp2_fast(u * 2.885390082f) + 1.f);
    return q < 0.0625f ? series : direct;
}

// A word's codes 0, 1 as the halves lo and codes 2, 3 as hi. The int8 codes come
// with their top bit flipped (u = code + 128): the half 0x6400 | u is 1024 + u.
template <bool INT8>
__device__ __forceinline__ void halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if (INT8) {
        const uint32_t x = __byte_perm(w, 0x64646464u, 0x4140), y = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 off = __half2half2(__ushort_as_half(0x6480));
        const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&x), off);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&y), off);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

// The transpose of an 8 x 8 matrix of halves held in the warp's fragment layout.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool INT8>
__device__ __forceinline__ uint32_t flip(uint32_t w) {
    return INT8 ? w ^ 0x80808080u : w;
}

// The tiles that some query in [q_lo, q_hi] of a sequence of `len` tokens sees:
// up to kMaxTerms disjoint runs, ascending. Returns the number of tiles.
__device__ __forceinline__ int seen_tiles(const MaskDnf& dnf, int64_t q_lo, int64_t q_hi, int64_t len, int* first,
                                          int* last, int* runs) {
    int n = 0, total = 0;
    for (int t = 0; t < dnf.n_terms; ++t) {
        int64_t lo, hi, unused;
        term_interval(dnf, t, q_lo, 0, len - 1, 0, 0, lo, unused);  // intervals move up with the query
        term_interval(dnf, t, q_hi, 0, len - 1, 0, 0, unused, hi);
        if (lo > hi) continue;
        int a = static_cast<int>(lo / kTileTokens), b = static_cast<int>(hi / kTileTokens);
        // into the sorted list, with every run that it meets
        int at = 0, keep = 0;
        int i = 0;
        while (i < n && last[i] < a) ++i;
        at = i;
        while (i < n && first[i] <= b) {
            a = min(a, first[i]);
            b = max(b, last[i]);
            total -= last[i] - first[i] + 1;
            ++i;
        }
        keep = n - i;
        if (i > at) {  // `i - at` runs become one
            for (int j = 0; j < keep; ++j) first[at + 1 + j] = first[i + j], last[at + 1 + j] = last[i + j];
        } else {
            for (int j = keep; j > 0; --j) first[at + j] = first[at + j - 1], last[at + j] = last[at + j - 1];
        }
        first[at] = a;
        last[at] = b;
        total += b - a + 1;
        n = at + 1 + keep;
    }
    *runs = n;
    return total;
}

struct PagedSeq {
    int slot;           // row of the page table, -1: none (length 0)
    int64_t len;
    int64_t q0;         // the first query token
    int count;          // queries
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int i) {
    PagedSeq s;
    s.slot = p.seqs[i];
    int64_t q0 = i, q1 = i + 1;
    if (p.cu != nullptr) {
        q0 = p.cu[i];
        q1 = p.cu[i + 1];
        if (q0 < 0 || q1 < q0 || q1 > p.T) {
            set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);
            q1 = q0;
        }
    }
    s.q0 = q0;
    s.count = static_cast<int>(q1 - q0);
    s.len = 0;
    if (s.slot < 0 || s.slot >= p.c.max_seqs) {
        if (s.slot != -1) set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
        s.slot = -1;
    } else {
        const int64_t len = p.c.seq_lens[s.slot];
        if (len < 0 || len > seq_capacity(p.c))
            set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
        else
            s.len = len;
    }
    return s;
}

// A sequence and the tiles that its queries see.
struct PagedPlan {
    PagedSeq s;
    int tiles, runs;
    int first[kMaxTerms], last[kMaxTerms];
};

// What the blocks need of the sequence that they work on.
struct PagedSeqShared {
    PagedSeq s;
    int64_t weight;  // of all its units
    int tiles;
    int first[kMaxTerms], last[kMaxTerms];          // runs of seen tiles
    int32_t clean_lo[kMaxTerms], clean_hi[kMaxTerms];  // keys that every query sees, for each term
};

// A unit weighs its tiles and what it costs to begin and end one, in tiles. A
// sequence without a key still has one (empty) tile, which writes its rows.
constexpr int kUnitCost = 10;  // (6, 10, 16: ragged batch of 64 up to 16k 195, 194, 197 us; 4 + 1024 visible of 64 up to 32k 46.7, 46.0, 46.8)
template <int ROWS>
__device__ __forceinline__ int64_t paged_weight(const PagedParams& p, const PagedSeq& s, int tiles) {
    if (s.count == 0) return 0;
    const int64_t row_tiles = (static_cast<int64_t>(s.count) * p.group + ROWS - 1) / ROWS;
    return row_tiles * p.c.heads * (max(tiles, 1) + kUnitCost);
}

// MODS: 0 none, 1 soft-cap, 2 ALiBi with or without soft-cap.
template <int D, bool INT8, int NT, int MODS>
__global__ void __launch_bounds__(32 * PagedShape<D, NT>::kWarps, PagedShape<D, NT>::kBlocks)
    paged_attention_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ MaskDnf dnf,
                           const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using Shape = PagedShape<D, NT>;
    constexpr int kWarps = Shape::kWarps, kBlockThreads = 32 * kWarps;
    constexpr int kSteps = D / 16;   // MMA steps over the head dimension
    constexpr int kChunks = D / 64;  // 16-byte pieces of a K row that one lane holds
    constexpr int kOut = D / 16;     // output tiles of 16 columns of V
    constexpr int kRows = 8 * NT;
    constexpr bool kQShared = NT > 1;  // q's fragments in shared memory, not registers
    constexpr float kLog2e = 1.4426950408889634f;
    constexpr float kLn2 = 0.6931471805599453f;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bars[kWarps * 2 * Shape::kDeep];
    __shared__ long long s_scan[kWarps];
    __shared__ long long s_off;
    __shared__ int s_i;
    __shared__ PagedSeqShared s_seq;
    const KvCache& c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;");  // the combining kernel may take its place and wait for this one's end
    uint8_t* const smem = smem_raw + (1024u - (shared_addr(smem_raw) & 1023u)) % 1024u;  // (the swizzle's period)
    const uint32_t bars = shared_addr(s_bars) + warp * 2 * Shape::kDeep * 8;
    if (lane < 2 * Shape::kDeep) bar_init(bars + lane * 8);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&k_map)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&v_map)) : "memory");
    }

    // What the stream's earlier kernels wrote is there. (Plain loads below, no __ldg: these data may be written while this
    // kernel waits here, and only loads that are not taken for constant stay behind the wait.)
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- this block's share of all tiles
    const int per_thread = (p.n + kBlockThreads - 1) / kBlockThreads;
    const int i_lo = min(p.n, tid * per_thread), i_hi = min(p.n, i_lo + per_thread);
    auto plan = [&](int i, PagedPlan& d) {  // returns the sequence's weight
        d.s = paged_seq(p, i);
        d.tiles = seen_tiles(dnf, d.s.len - d.s.count, d.s.len - 1, d.s.len, d.first, d.last, &d.runs);
        return paged_weight<kRows>(p, d.s, d.tiles);
    };
    auto describe = [&](const PagedPlan& d) {  // for the whole block
        s_seq.s = d.s;
        s_seq.tiles = d.tiles;
        s_seq.weight = paged_weight<kRows>(p, d.s, d.tiles);
        for (int x = 0; x < d.runs; ++x) {
            s_seq.first[x] = d.first[x];
            s_seq.last[x] = d.last[x];
        }
        for (int x = 0; x < dnf.n_terms; ++x) {
            int64_t lo, hi, unused;  // (both within [-len, len])
            term_interval(dnf, x, d.s.len - 1, 0, d.s.len - 1, 0, 0, lo, unused);
            term_interval(dnf, x, d.s.len - d.s.count, 0, d.s.len - 1, 0, 0, unused, hi);
            s_seq.clean_lo[x] = static_cast<int32_t>(min(lo, static_cast<int64_t>(INT32_MAX)));
            s_seq.clean_hi[x] = static_cast<int32_t>(max(hi, static_cast<int64_t>(-1)));
        }
    };
    long long mine = 0;
    PagedPlan own;  // the thread's sequence, where there is one for each thread at most
    for (int i = i_lo; i < i_hi; ++i) mine += plan(i, own);
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long all = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        all += s_scan[w];
        if (w < warp) before += s_scan[w];
    }
    long long share = all <= static_cast<long long>(0xFFFFFFFFu - gridDim.x)
                          ? (static_cast<uint32_t>(all) + gridDim.x - 1) / gridDim.x
                          : (all + gridDim.x - 1) / gridDim.x;
    if (share < p.min_share) share = p.min_share;
    const long long begin = share * blockIdx.x, end = min(all, begin + share);
    if (begin < end && before <= begin && begin < before + mine) {
        long long off = begin - before;
        int i = i_lo;
        if (per_thread > 1) {
            for (; i < i_hi; ++i) {
                const long long w = plan(i, own);
                if (off < w) break;
                off -= w;
            }
        }
        s_i = i;
        s_off = off;
        describe(own);
    }
    if (tid == 0) p.heads_of_parts[blockIdx.x * 8] = 0;
    // rows behind the last sequence, or, against the conditions, in front of the first, belong to none: they see nothing
    if (p.cu != nullptr) {
        const int T = static_cast<int>(p.T), used = max(0, min(p.cu[p.n], T)), front = max(0, min(p.cu[0], used));
        if (front > 0) set_status(p.status, BSMT_ERR_DEVICE_PRECONDITION);
        for (int part = 0; part < 2; ++part) {
            const int64_t from = part == 0 ? used : 0, tokens = part == 0 ? T - used : front;
            if (tokens == 0) continue;
            const int64_t stride = static_cast<int64_t>(gridDim.x) * kBlockThreads;
            const int64_t rest = tokens * p.Hq;
            uint4* o = reinterpret_cast<uint4*>(p.out + from * p.Hq * D);
            for (int64_t x = static_cast<int64_t>(blockIdx.x) * kBlockThreads + tid; x < rest * (D / 8); x += stride)
                o[x] = make_uint4(0, 0, 0, 0);
            for (int64_t x = static_cast<int64_t>(blockIdx.x) * kBlockThreads + tid; x < rest; x += stride)
                p.lse[x / tokens * p.T + from + x % tokens] = -INFINITY;
        }
    }
    __syncthreads();
    if (begin >= end) return;

    int i = s_i;
    long long off = s_off, left = end - begin;
    bool first_segment = true;
    const uint32_t slots = shared_addr(smem) + warp * Shape::kWarpBytes;  // K of tile x, V of tile x, ...
    const float* const lane_scales = ((lane & 2) ? c.v_scale : c.k_scale) + static_cast<int64_t>(p.layer) * c.pages * c.heads;
    // The slots hold rows of D bytes whose 16-byte pieces the copy has swizzled: piece ^ row % 8 (D = 128), piece ^
    // row / 2 % 4 (D = 64). Token `slot_token(g)` of each 8 is the products' row g: the order in which neither the K
    // reads (rows g, pieces t) nor the V reads (rows 2 t and 2 t + 1, pieces g) meet a bank twice.
    auto slot_token = [](int x) {
        const int u = x >> 1;
        if (D == 128) return (x & 1) ? ((2 * u) ^ 4) | 1 : 2 * u;
        const int even = (u & 1) | (u >> 1) << 2;
        return (x & 1) ? even ^ 3 : even;
    };
    const int tok_g = slot_token(g);
    uint32_t k_at[kChunks], v_at[2];  // this lane's pieces of the first 8 rows
#pragma unroll
    for (int x = 0; x < kChunks; ++x) k_at[x] = tok_g * D + (D == 128 ? ((4 * x + t) ^ tok_g) * 16 : (t ^ (tok_g >> 1)) * 16);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int row = slot_token(2 * t + x);
        v_at[x] = row * D + (D == 128 ? (g ^ row) * 16 : ((g >> 1) ^ (row >> 1)) * 16 + (g & 1) * 8);
    }
    uint32_t bar_k = bars, parity = 0;  // the next tile's barriers (K, then V) and their phase
    uint32_t slot_k = slots;

    while (true) {
        const int len = static_cast<int>(s_seq.s.len);
        const int count = s_seq.s.count;
        const int seen = s_seq.tiles, tiles = max(seen, 1);
        const int64_t weight = s_seq.weight;
        const int32_t* table = c.page_table + static_cast<int64_t>(max(s_seq.s.slot, 0)) * c.max_pages;
        const int64_t rows_all = static_cast<int64_t>(count) * p.group;
        int unit = 0, in_unit = 0;  // in_unit: of the unit's weight, its cost first
        if (off != 0) {
            const long long u = off <= 0x7FFFFFFF ? static_cast<uint32_t>(off) / static_cast<uint32_t>(tiles + kUnitCost) : off / (tiles + kUnitCost);
            unit = static_cast<int>(u);
            in_unit = static_cast<int>(off - u * (tiles + kUnitCost));
        }
        int tile_row = unit / c.heads;
        int head = unit - tile_row * c.heads;

        while (off < weight && left > 0) {
            const int take = static_cast<int>(min(static_cast<long long>(tiles + kUnitCost - in_unit), left));
            const int t0 = max(0, in_unit - kUnitCost), t1 = max(0, in_unit + take - kUnitCost);
            off += take;
            left -= take;
            in_unit = 0;
            if (t1 == 0) break;  // (the share ends before the unit's first tile)
            const int64_t row0 = static_cast<int64_t>(tile_row) * kRows;  // the unit's first row
            const int64_t qi0 = rows_all < 0x7FFFFFFF ? static_cast<int64_t>(static_cast<uint32_t>(row0) / static_cast<uint32_t>(p.group))
                                                      : row0 / p.group;
            const int in_group = static_cast<int>(row0 - qi0 * p.group);  // row0 = qi0 * group + in_group

            // ---- pipeline over this warp's tiles
            const int stop = min(t1, seen);
            int run = -1, run_end = 0, run_off = 0;  // the run that the next tile to load lies in: its last ordinal + 1, and
                                                     // its first tile less its first ordinal
            auto tile_of = [&](int ord) -> int {  // first token of the unit's tile `ord`; -1: none
                if (ord >= stop) return -1;
                while (ord >= run_end) {
                    ++run;
                    run_off = s_seq.first[run] - run_end;
                    run_end += s_seq.last[run] - s_seq.first[run] + 1;
                }
                return (ord + run_off) * kTileTokens;
            };
            auto page_at = [&](int tok) -> int {  // page of a token; -1: behind the sequence
                if (tok < 0 || tok >= len) return -1;
                return table[tok >> c.page_shift];
            };
            // the page of the tile's second half: another one with pages of 16
            auto second_page = [&](int tok, int first) -> int { return c.page == 16 ? page_at(tok < 0 ? -1 : tok + 16) : first; };
            int next_ord = t0 + warp;  // (after the first loads: the tile that find_next has found)
            int next_tok = -1, next_a = -1, next_b = -1;
            int tok_q[Shape::kDeep];      // first tokens of the tiles on their way
            int row_a[Shape::kDeep], row_b[Shape::kDeep];  // their rows in the pools
            float scale_q[Shape::kDeep];  // lane % 4: k_scale of the tile's halves of 16 tokens, v_scale of them
            const int no_row = c.layers * c.pages * c.heads * c.page;  // behind the pool: a load gives zeros
            auto load = [&](const CUtensorMap* map, uint32_t slot, uint32_t bar, int ra, int rb) {
                if (lane == 0) {
                    bar_expect(bar, Shape::kSlot);
                    load_rows(slot, map, ra, bar);
                    if (c.page == 16) load_rows(slot + 16 * D, map, rb, bar);
                }
            };
            // Finds the rows of the next tile and starts its K load; its V load follows once that slot is free.
            auto begin_tile = [&](int x, uint32_t slot, uint32_t bar) {
                tok_q[x] = next_tok;
                if (next_tok >= 0) {
                    const bool ok_a = next_a >= 0 && next_a < c.pages, ok_b = next_b >= 0 && next_b < c.pages;
                    if ((!ok_a || (!ok_b && next_tok + 16 < len)) && lane == 0) set_status(p.status, BSMT_ERR_DEVICE_BOUNDS);
                    row_a[x] = ok_a ? ((p.layer * c.pages + next_a) * c.heads + head) * c.page + (next_tok & (c.page - 1)) : no_row;
                    row_b[x] = ok_b ? ((p.layer * c.pages + next_b) * c.heads + head) * c.page + ((next_tok + 16) & (c.page - 1)) : no_row;
                    scale_q[x] = ((lane & 1) ? ok_b : ok_a) ? lane_scales[static_cast<int64_t>((lane & 1) ? next_b : next_a) * c.heads + head] : 0.f;
                    load(&k_map, slot, bar, row_a[x], row_b[x]);
                }
            };
            auto find_next = [&](int tok, int a, int b) {
                next_tok = tok;
                next_a = a;
                next_b = b;
            };
            uint4 q_raw[NT][kChunks][2];
            {
                int first_tok[Shape::kDeep + 1], first_a[Shape::kDeep + 1], first_b[Shape::kDeep + 1];  // (read together)
#pragma unroll
                for (int x = 0; x <= Shape::kDeep; ++x) {
                    first_tok[x] = tile_of(next_ord + x * kWarps);
                    first_a[x] = page_at(first_tok[x]);
                    first_b[x] = second_page(first_tok[x], first_a[x]);
                }
                // q's rows g of each 8, read meanwhile
#pragma unroll
                for (int r = 0; r < NT; ++r) {
                    const int row = 8 * r + g;
                    const bool valid = row0 + row < rows_all;
                    const int up_q = static_cast<int>(static_cast<uint32_t>(in_group + row) / static_cast<uint32_t>(p.group));
                    const int64_t qi = valid ? qi0 + up_q : 0;
                    const int hq = head * p.group + (valid ? in_group + row - up_q * p.group : 0);
                    const uint4* src = reinterpret_cast<const uint4*>(p.q + ((s_seq.s.q0 + qi) * p.Hq + hq) * D + 16 * t);
#pragma unroll
                    for (int x = 0; x < kChunks; ++x) {
                        q_raw[r][x][0] = valid ? src[8 * x] : make_uint4(0, 0, 0, 0);
                        q_raw[r][x][1] = valid ? src[8 * x + 1] : make_uint4(0, 0, 0, 0);
                    }
                }
                uint32_t slot = slot_k, bar = bar_k;
#pragma unroll
                for (int x = 0; x < Shape::kDeep; ++x) {
                    next_tok = first_tok[x];
                    next_a = first_a[x];
                    next_b = first_b[x];
                    begin_tile(x, slot, bar);
                    if (tok_q[x] >= 0) load(&v_map, slot + Shape::kSlot, bar + 8, row_a[x], row_b[x]);
                    slot = slot + 2 * Shape::kSlot == slots + Shape::kWarpBytes ? slots : slot + 2 * Shape::kSlot;
                    bar = bar + 16 == bars + 16 * Shape::kDeep ? bars : bar + 16;
                }
                find_next(first_tok[Shape::kDeep], first_a[Shape::kDeep], first_b[Shape::kDeep]);
                next_ord += Shape::kDeep * kWarps;
            }

            // ---- q in halves; what the softmax needs of rows 2 t and 2 t + 1
            uint32_t qf[kQShared ? 1 : NT][kSteps][2];
            float qs[NT][2], slope[MODS == 2 ? NT : 1][2];
            auto pos_of = [&](int r, int y) {  // position of the query of row 8 r + 2 t + y
                return len - count + static_cast<int>(qi0) +
                       static_cast<int>(static_cast<uint32_t>(in_group + 8 * r + 2 * t + y) / static_cast<uint32_t>(p.group));
            };
            int pos[MODS == 2 ? NT : 1][2];
            const uint32_t q_smem = shared_addr(smem) + Shape::kQ + lane * 8;
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                uint32_t w[kChunks][8];
#pragma unroll
                for (int x = 0; x < kChunks; ++x) {
                    const uint4 a = q_raw[r][x][0], b = q_raw[r][x][1];
                    w[x][0] = a.x, w[x][1] = a.y, w[x][2] = a.z, w[x][3] = a.w;
                    w[x][4] = b.x, w[x][5] = b.y, w[x][6] = b.z, w[x][7] = b.w;
                }
                uint32_t most = 0;
#pragma unroll
                for (int x = 0; x < kChunks; ++x)
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const uint32_t a = w[x][y] & 0x7FFFu, b = w[x][y] >> 16 & 0x7FFFu;
                        most = max(most, max(a < 0x7F80u ? a : 0u, b < 0x7F80u ? b : 0u));
                    }
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                // largest value to [2^14, 2^15): the row's small values keep their bits, too
                const int e = max(static_cast<int>(most >> 7) - 127, -100) - 14;
                const float row_scale = exp2i(e) * p.scale * (MODS != 0 ? 1.f : kLog2e);
                const float up = exp2i(-e);
#pragma unroll
                for (int x = 0; x < kChunks; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t u[2];
#pragma unroll
                        for (int z = 0; z < 2; ++z)
                            u[z] = pack_half2(__uint_as_float(w[x][2 * y + z] << 16) * up,
                                              __uint_as_float(w[x][2 * y + z] & 0xFFFF0000u) * up);
                        if (!kQShared) {
                            qf[r][4 * x + y][0] = u[0], qf[r][4 * x + y][1] = u[1];
                        } else if (warp == r) {
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(q_smem + (r * kSteps + 4 * x + y) * 256),
                                         "r"(u[0]), "r"(u[1])
                                         : "memory");
                        }
                    }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    qs[r][y] = __shfl_sync(0xFFFFFFFFu, row_scale, (2 * t + y) * 4);
                    if (MODS == 2) {
                        const int col = 8 * r + 2 * t + y;
                        pos[r][y] = pos_of(r, y);
                        slope[r][y] = 0.f;
                        if (row0 + col < rows_all) {
                            const int h = head * p.group + in_group + col - (pos[r][y] - (len - count) - static_cast<int>(qi0)) * p.group;
                            slope[r][y] = p.slopes != nullptr
                                              ? p.slopes[h]
                                              : exp2f(-8.f * static_cast<float>(p.alibi_h0 + h + 1) / static_cast<float>(p.alibi_heads));
                        }
                    }
                }
            }
            if (kQShared) __syncthreads();

            const int clean_lo = s_seq.clean_lo[0], clean_hi = s_seq.clean_hi[0];
            float o[NT][kOut][4];
            float m[NT][2], mo[NT][2], l[NT][2];
#pragma unroll
            for (int r = 0; r < NT; ++r) {
#pragma unroll
                for (int y = 0; y < 2; ++y) m[r][y] = mo[r][y] = -INFINITY, l[r][y] = 0.f;
#pragma unroll
                for (int x = 0; x < kOut; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[r][x][y] = 0.f;
            }

            for (int ord = t0 + warp; ord < t1; ord += kWarps) {
                const int tok = tok_q[0];
                if (tok >= 0) {
                    // s[r][h][2 z + y]: token 16 h + 8 z + tok_g, row 8 r + 2 t + y
                    float s[NT][2][4];
#pragma unroll
                    for (int r = 0; r < NT; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int y = 0; y < 4; ++y) s[r][h][y] = 0.f;
                    bar_wait(bar_k, parity, p.status);
#pragma unroll
                    for (int x = 0; x < kChunks; ++x) {
                        uint32_t kw[4][4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint4 v = lds128(slot_k + k_at[x] + j * 8 * D);
                            kw[j][0] = flip<INT8>(v.x), kw[j][1] = flip<INT8>(v.y), kw[j][2] = flip<INT8>(v.z), kw[j][3] = flip<INT8>(v.w);
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            uint32_t b[NT][2];
#pragma unroll
                            for (int r = 0; r < NT; ++r) {
                                if (!kQShared) {
                                    b[r][0] = qf[r][4 * x + y][0], b[r][1] = qf[r][4 * x + y][1];
                                } else {
                                    const uint2 v = lds64(q_smem + (r * kSteps + 4 * x + y) * 256);
                                    b[r][0] = v.x, b[r][1] = v.y;
                                }
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t a[4];  // tokens g, g + 8; codes 0, 1 then 2, 3
                                halves<INT8>(kw[2 * h][y], a[0], a[2]);
                                halves<INT8>(kw[2 * h + 1][y], a[1], a[3]);
#pragma unroll
                                for (int r = 0; r < NT; ++r) mma16816(s[r][h], a, b[r][0], b[r][1]);
                            }
                        }
                    }
                    const float ks[2] = {__shfl_sync(0xFFFFFFFFu, scale_q[0], 0), __shfl_sync(0xFFFFFFFFu, scale_q[0], 1)};
                    const float vs[2] = {__shfl_sync(0xFFFFFFFFu, scale_q[0], 2), __shfl_sync(0xFFFFFFFFu, scale_q[0], 3)};
                    const float ev[2] = {__log2f(fmaxf(vs[0], 0x1p-120f)), __log2f(fmaxf(vs[1], 0x1p-120f))};  // (so that m - mo is at most 127)

                    // which keys the rows see
                    bool clean = clean_lo <= tok && tok + kTileTokens - 1 <= clean_hi;
                    for (int x = 1; x < dnf.n_terms; ++x)
                        clean = clean || (s_seq.clean_lo[x] <= tok && tok + kTileTokens - 1 <= s_seq.clean_hi[x]);
                    uint32_t bits[NT][2];
                    if (!clean) {
#pragma unroll
                        for (int r = 0; r < NT; ++r)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int at = pos_of(r, y);
                                bits[r][y] = 0;
                                for (int x = 0; x < dnf.n_terms; ++x) {
                                    int64_t lo, hi;
                                    term_interval(dnf, x, at, 0, len - 1, 0, 0, lo, hi);
                                    bits[r][y] |= range_bits(lo, hi, tok);
                                }
                            }
                    }
                    if (MODS == 1) {
                        // cap * tanh(z / cap), in units of log2. Up to a cap of 64 the exponential's form alone: its error
                        // is cap * 2^-23, below a score's own, and all factors go into one (at most the largest float, so
                        // that a product q . k of 0 stays 0). Beyond, a score may be small beside the cap, and 1 / cap
                        // times the row's and the page's scales too small for a float: z comes first.
#pragma unroll
                        for (int r = 0; r < NT; ++r)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float u[2] = {qs[r][0] * ks[h], qs[r][1] * ks[h]};
                                if (p.cap <= 64.f) {
                                    const float cap2 = p.cap * kLog2e;
                                    const float w[2] = {fminf(u[0] * p.cap_inv, FLT_MAX), fminf(u[1] * p.cap_inv, FLT_MAX)};
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        s[r][h][e] = fmaf(-2.f * cap2, rcp_fast(exp2_fast(s[r][h][e] * w[e & 1]) + 1.f), cap2);
                                } else {
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        s[r][h][e] = p.cap * tanh_fast(s[r][h][e] * u[e & 1] * p.cap_inv) * kLog2e;
                                }
                            }
                    } else if (MODS == 2) {
                        const int rel = tok - pos[0][0] + tok_g;
#pragma unroll
                        for (int r = 0; r < NT; ++r)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int y = e & 1;
                                    float z = s[r][h][e] * (qs[r][y] * ks[h]);
                                    const float bias = slope[r][y] * static_cast<float>(rel + 16 * h + 8 * (e >> 1) - (pos[r][y] - pos[0][0]));
                                    if (p.alibi_first) z += bias;
                                    if (p.softcap) z = p.cap * tanh_fast(z / p.cap);
                                    if (!p.alibi_first) z += bias;
                                    s[r][h][e] = z * kLog2e;
                                }
                    }
                    if (!clean) {
#pragma unroll
                        for (int r = 0; r < NT; ++r)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (!(bits[r][e & 1] >> (16 * h + 8 * (e >> 1) + tok_g) & 1u)) s[r][h][e] = -INFINITY;
                    }

                    // The references stay while no score passes one by more than kLazy: then the lanes need not
                    // agree on a maximum, and O is not rescaled.
                    float f[NT][2][2];  // a score is s * f, f > 0 (a scale of 0 belongs to codes of 0)
                    bool grows = false;
#pragma unroll
                    for (int r = 0; r < NT; ++r)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                f[r][y][h] = MODS != 0 ? 1.f : fmaxf(qs[r][y] * ks[h], 1e-37f);
                                const float top = fmaxf(s[r][h][y], s[r][h][2 + y]) * f[r][y][h];
                                grows = grows || top > m[r][y] + kLazy || top + ev[h] > mo[r][y] + (kLazy + kRoom);
                            }
                    if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
                        for (int r = 0; r < NT; ++r) {
                            float ao[2];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                float top[2];  // of each 16 tokens
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    top[h] = fmaxf(s[r][h][y], s[r][h][2 + y]) * f[r][y][h];
                                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], 4));
                                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], 8));
                                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], 16));
                                }
                                const float mn = fmaxf(m[r][y], fmaxf(top[0], top[1]));
                                const float mon = fmaxf(mo[r][y], fmaxf(top[0] + ev[0], top[1] + ev[1]) - kRoom);
                                const float ref = mn == -INFINITY ? 0.f : mn, refo = mon == -INFINITY ? 0.f : mon;
                                l[r][y] *= exp2_fast(m[r][y] - ref);
                                ao[y] = exp2_fast(mo[r][y] - refo);
                                m[r][y] = mn;
                                mo[r][y] = mon;
                            }
#pragma unroll
                            for (int x = 0; x < kOut; ++x)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[r][x][e] *= ao[e & 1];
                        }
                    }
                    // every lane has used the K slot (the vote above needed its scores): the tile kDeep further goes there
#pragma unroll
                    for (int x = 0; x + 1 < Shape::kDeep; ++x) {
                        tok_q[x] = tok_q[x + 1];
                        row_a[x] = row_a[x + 1];
                        row_b[x] = row_b[x + 1];
                        scale_q[x] = scale_q[x + 1];
                    }
                    begin_tile(Shape::kDeep - 1, slot_k, bar_k);
                    next_ord += kWarps;
                    const int found = tile_of(next_ord);
                    const int found_a = page_at(found);
                    find_next(found, found_a, second_page(found, found_a));
                    uint32_t pb[NT][2][2];
#pragma unroll
                    for (int r = 0; r < NT; ++r) {
                        const float ref[2] = {m[r][0] == -INFINITY ? 0.f : m[r][0], m[r][1] == -INFINITY ? 0.f : m[r][1]};
                        // 2^(m - mo), 0 for a row that has seen nothing
                        const float shift[2] = {m[r][0] == -INFINITY ? 0.f : exp2_fast(m[r][0] - mo[r][0]),
                                                m[r][1] == -INFINITY ? 0.f : exp2_fast(m[r][1] - mo[r][1])};
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                float e[2];
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    e[y] = exp2_fast(MODS != 0 ? s[r][h][2 * z + y] - ref[y] : fmaf(s[r][h][2 * z + y], f[r][y][h], -ref[y]));
                                    l[r][y] += e[y];
                                }
                                // P to a half: an error of 2^-12 of each term down to 2^-21 of the largest, of 2^-32 of the
                                // largest for smaller ones, below the output's bf16 rounding for up to 2^22 keys
                                pb[r][h][z] = transpose8x8(pack_half2(e[0] * (vs[h] * shift[0]), e[1] * (vs[h] * shift[1])));
                            }
                    }

                    bar_wait(bar_k + 8, parity, p.status);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // 16 tokens
                        uint32_t vw[4][D / 32];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t a = slot_k + Shape::kSlot + v_at[x & 1] + (16 * h + 8 * (x >> 1)) * D;
                            if (D == 128) {
                                const uint4 v = lds128(a);
                                vw[x][0] = v.x, vw[x][1] = v.y, vw[x][D / 32 - 2] = v.z, vw[x][D / 32 - 1] = v.w;
                            } else {
                                const uint2 v = lds64(a);
                                vw[x][0] = v.x, vw[x][1] = v.y;
                            }
                        }
                        // 4 x 4 bytes: token-major words -> for each column of V its four tokens; tile 2 w + b has
                        // columns 4 w + 2 b (rows g) and 4 w + 2 b + 1 (rows g + 8) of the lane's D / 8
                        auto columns = [&](const uint32_t w0, const uint32_t w1, const uint32_t w2, const uint32_t w3, int b, uint32_t a[4]) {
                            halves<INT8>(__byte_perm(w0, w1, b ? 0x7362 : 0x5140), a[0], a[1]);
                            halves<INT8>(__byte_perm(w2, w3, b ? 0x7362 : 0x5140), a[2], a[3]);
                        };
                        if (!INT8 && !clean) {
                            // 0 * NaN: a NaN code that some row does not see must not reach that row. Rare
                            // (NaN values in a tile on the mask's edge): the codes become 0 here, and rows
                            // that see one get NaN from a product of NaN indicators and visibility.
                            uint32_t found = 0;
#pragma unroll
                            for (int x = 0; x < 4; ++x)
#pragma unroll
                                for (int y = 0; y < D / 32; ++y) found |= ((vw[x][y] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                            if (__any_sync(0xFFFFFFFFu, found != 0u)) {
                                uint32_t see[NT][2];
#pragma unroll
                                for (int r = 0; r < NT; ++r)
#pragma unroll
                                    for (int z = 0; z < 2; ++z) {
                                        const int at = 16 * h + 8 * z + tok_g;
                                        see[r][z] = transpose8x8((bits[r][0] >> at & 1u) * 0x3C00u | (bits[r][1] >> at & 1u) * 0x3C000000u);
                                    }
#pragma unroll
                                for (int w = 0; w < D / 32; ++w) {
                                    uint32_t ind[4];
#pragma unroll
                                    for (int x = 0; x < 4; ++x) {
                                        const uint32_t nan = ((((vw[x][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu;
                                        vw[x][w] &= ~nan;
                                        ind[x] = nan & 0x38383838u;  // e4m3 1.0
                                    }
#pragma unroll
                                    for (int b = 0; b < 2; ++b) {
                                        uint32_t a[4];
                                        columns(ind[0], ind[1], ind[2], ind[3], b, a);
#pragma unroll
                                        for (int r = 0; r < NT; ++r) {
                                            float hit[4] = {0.f, 0.f, 0.f, 0.f};
                                            mma16816(hit, a, see[r][0], see[r][1]);
#pragma unroll
                                            for (int z = 0; z < 4; ++z)
                                                if (hit[z] > 0.f) o[r][2 * w + b][z] = __int_as_float(0x7FFFFFFF);
                                        }
                                    }
                                }
                            }
                        }
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            const uint32_t w0 = flip<INT8>(vw[0][w]), w1 = flip<INT8>(vw[1][w]), w2 = flip<INT8>(vw[2][w]),
                                           w3 = flip<INT8>(vw[3][w]);
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                uint32_t a[4];
                                columns(w0, w1, w2, w3, b, a);
#pragma unroll
                                for (int r = 0; r < NT; ++r) mma16816(o[r][2 * w + b], a, pb[r][h][0], pb[r][h][1]);
                            }
                        }
                    }
                }
                if (tok >= 0) {
                    __syncwarp();  // every lane has read the V slot
                    if (tok_q[Shape::kDeep - 1] >= 0)
                        load(&v_map, slot_k + Shape::kSlot, bar_k + 8, row_a[Shape::kDeep - 1], row_b[Shape::kDeep - 1]);
                    slot_k += 2 * Shape::kSlot;
                    bar_k += 16;
                    if (slot_k == slots + Shape::kWarpBytes) {
                        slot_k = slots;
                        bar_k = bars;
                        parity ^= 1;
                    }
                }
            }

            // ---- the four warps' parts of the segment become one
            __syncthreads();
            float* s_o = reinterpret_cast<float*>(smem);               // [warp][row][kPitch]
            float* s_m = s_o + kWarps * kRows * Shape::kPitch;    // [warp][row][4]
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float sum = l[r][y];
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
                    const int row = warp * kRows + 8 * r + 2 * t + y;
                    if (g == 0) *reinterpret_cast<float4*>(s_m + row * 4) = make_float4(m[r][y], mo[r][y], sum, 0.f);
                    // tile x holds columns g * (D / 8) + 2 x and + 1 of V
#pragma unroll
                    for (int x = 0; x < kOut; x += 2)
                        *reinterpret_cast<float4*>(s_o + row * Shape::kPitch + g * (D / 8) + 2 * x) =
                            make_float4(o[r][x][y], o[r][x][2 + y], o[r][x + 1][y], o[r][x + 1][2 + y]);
                }
            __syncthreads();
            const bool whole = t0 == 0 && t1 == tiles;
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (first_segment ? 0 : 1);
            if (!whole && t0 == 0 && tid == 0) {
                int32_t* hd = p.heads_of_parts + blockIdx.x * 8;
                hd[1] = first_segment ? 0 : 1;
                hd[2] = static_cast<int32_t>(s_seq.s.q0);
                hd[3] = count;
                hd[4] = head;
                hd[5] = static_cast<int32_t>(row0 & 0xFFFFFFFF);
                hd[6] = static_cast<int32_t>(row0 >> 32);
                hd[0] = 1 + static_cast<int32_t>((tiles - t1 + share - 1) / share);
            }
            for (int x = tid; x < kRows * (D / 4); x += kBlockThreads) {
                const int row = x / (D / 4), d = (x % (D / 4)) * 4;
                if (row0 + row >= rows_all) continue;
                float4 sm[kWarps];
                float mm = -INFINITY, mmo = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    sm[w] = *reinterpret_cast<const float4*>(s_m + (w * kRows + row) * 4);
                    mm = fmaxf(mm, sm[w].x);
                    mmo = fmaxf(mmo, sm[w].y);
                }
                const float ref = mm == -INFINITY ? 0.f : mm, refo = mmo == -INFINITY ? 0.f : mmo;
                float sum = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    sum += sm[w].z * exp2_fast(sm[w].x - ref);
                    const float f = exp2_fast(sm[w].y - refo);
                    const float4 v = *reinterpret_cast<const float4*>(s_o + (w * kRows + row) * Shape::kPitch + d);
                    acc.x = fmaf(f, v.x, acc.x);
                    acc.y = fmaf(f, v.y, acc.y);
                    acc.z = fmaf(f, v.z, acc.z);
                    acc.w = fmaf(f, v.w, acc.w);
                }
                if (whole) {
                    const int up_q = static_cast<int>(static_cast<uint32_t>(in_group + row) / static_cast<uint32_t>(p.group));
                    const int64_t token = s_seq.s.q0 + qi0 + up_q;
                    const int hq = head * p.group + in_group + row - up_q * p.group;
                    // (a NaN sum is a row whose scores are NaN)
                    const float f = sum == 0.f ? 0.f : exp2_fast(refo + kRoom - ref) / sum;
                    const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * kRoomInv * f, acc.y * kRoomInv * f),
                                         b = __floats2bfloat162_rn(acc.z * kRoomInv * f, acc.w * kRoomInv * f);
                    *reinterpret_cast<uint2*>(p.out + (token * p.Hq + hq) * D + d) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
                    if (d == 0) p.lse[static_cast<int64_t>(hq) * p.T + token] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
                } else {
                    *reinterpret_cast<float4*>(p.part_o + (slot * kRows + row) * D + d) = acc;
                    if (d == 0) *reinterpret_cast<float4*>(p.part_m + (slot * kRows + row) * 4) = make_float4(mm, mmo, sum, 0.f);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the slots take copies again
            __syncthreads();
            first_segment = false;
            if (++head == c.heads) {
                head = 0;
                ++tile_row;
            }
        }
        // ---- the next sequence that has queries
        off = 0;
        if (left <= 0) break;
        while (true) {
            if (++i >= p.n) return;
            if (per_thread == 1) {
                if (tid == i) describe(own);
            } else if (tid == 0) {
                plan(i, own);
                describe(own);
            }
            __syncthreads();
            if (s_seq.weight != 0) break;
            __syncthreads();  // every thread has read it before the next description is written over it
        }
    }
}

// Joins the parts of the units that share boundaries cut: a unit that begins in
// block b's share ends in that of block b + parts - 1, and its later parts are those
// blocks' first. A block has four rows: a warp for each, or, with many parts, all
// warps on one row after another, each taking every fourth part.
template <int D, int ROWS>
__global__ void __launch_bounds__(32 * kCombineWarps) paged_combine_kernel(const __grid_constant__ PagedParams p) {
    constexpr float kLn2 = 0.6931471805599453f;
    constexpr int kPer = D / 32;  // columns of one lane
    constexpr int kFew = 16;
    __shared__ float s_o[kCombineWarps][D];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4* hd = reinterpret_cast<const int4*>(p.heads_of_parts + blockIdx.x * 8);
    const int4 h0 = hd[0];
    const int parts = h0.x;
    if (parts == 0) return;
    const int4 h1 = hd[1];
    const int64_t row0 = static_cast<int64_t>(static_cast<uint32_t>(h1.y)) | static_cast<int64_t>(h1.z) << 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool few = parts <= kFew;
    for (int x = few ? warp : 0; x < kCombineWarps; x += few ? kCombineWarps : 1) {
        const int in_tile = blockIdx.y * kCombineWarps + x;
        const int64_t row = row0 + in_tile;
        if (row >= static_cast<int64_t>(h0.w) * p.group) return;  // (uniform over the warps that share a row)
        auto slot_of = [&](int j) -> int64_t {
            return (2 * (static_cast<int64_t>(blockIdx.x) + j) + (j == 0 ? h0.y : 0)) * ROWS + in_tile;
        };
        float m = -INFINITY, mo = -INFINITY;
        for (int j = lane; j < parts; j += 32) {
            const float4 v = *reinterpret_cast<const float4*>(p.part_m + slot_of(j) * 4);
            m = fmaxf(m, v.x);
            mo = fmaxf(mo, v.y);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            mo = fmaxf(mo, __shfl_xor_sync(0xFFFFFFFFu, mo, d));
        }
        const float ref = m == -INFINITY ? 0.f : m, refo = mo == -INFINITY ? 0.f : mo;
        float sum = 0.f;
        for (int j = lane; j < parts; j += 32) {
            const float4 v = *reinterpret_cast<const float4*>(p.part_m + slot_of(j) * 4);
            sum += v.z * exp2_fast(v.x - ref);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        float acc[kPer];
#pragma unroll
        for (int y = 0; y < kPer; ++y) acc[y] = 0.f;
#pragma unroll 8
        for (int j = few ? 0 : warp; j < parts; j += few ? 1 : kCombineWarps) {
            const int64_t s = slot_of(j);
            const float f = exp2_fast(p.part_m[s * 4 + 1] - refo);
            const Pack<float, kPer> v = *reinterpret_cast<const Pack<float, kPer>*>(p.part_o + s * D + lane * kPer);
#pragma unroll
            for (int y = 0; y < kPer; ++y) acc[y] = fmaf(f, v.v[y], acc[y]);
        }
        const int64_t qi = row / p.group;
        const int hq = h1.x * p.group + static_cast<int>(row - qi * p.group);
        const int64_t token = h0.z + qi;
        if (!few) {
            __syncthreads();
#pragma unroll
            for (int y = 0; y < kPer; ++y) s_o[warp][lane * kPer + y] = acc[y];
            __syncthreads();
#pragma unroll
            for (int y = 0; y < kPer; ++y) {
                acc[y] = 0.f;
#pragma unroll
                for (int w = 0; w < kCombineWarps; ++w) acc[y] += s_o[w][lane * kPer + y];
            }
            if (warp != 0) continue;
        }
        const float f = sum == 0.f ? 0.f : exp2_fast(refo + kRoom - ref) / sum;
        Pack<__nv_bfloat16, kPer> r;
#pragma unroll
        for (int y = 0; y < kPer; ++y) r.v[y] = __float2bfloat16_rn(acc[y] * kRoomInv * f);
        *reinterpret_cast<Pack<__nv_bfloat16, kPer>*>(p.out + (token * p.Hq + hq) * D + lane * kPer) = r;
        if (lane == 0) p.lse[static_cast<int64_t>(hq) * p.T + token] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
    }
}

}  // namespace bsmt
