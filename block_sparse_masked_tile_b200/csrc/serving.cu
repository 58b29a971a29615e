// libbsmt: rotary positions, the 8-bit paged cache, and attention over it (the
// entry points of include/bsmt_serving.h, that a server calls beside flex_attention).
//
// Host side: argument checks and launches. Nothing here allocates device memory
// and nothing synchronizes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>

#include "bsmt_serving.h"
#include "host_common.h"
#include "kv_cache.cuh"
#include "paged_attn.cuh"
#include "rotary.cuh"

using namespace bsmt_host;

namespace {

// Kernels whose shared memory size has been raised on a device.
std::mutex g_set_mu;
bool g_paged_set[64][36] = {{false}};
bool g_compact_set[64] = {false};

constexpr int kMaxSeqs = 1 << 18;  // one bit each in the page planners' shared memory
constexpr int kMaxPartBlocks = 160 * 3;        // of paged attention, three an SM
constexpr int kMaxPartRows = 160 * 2 * 32;      // query rows of all its blocks: two of 32 or three of 16 an SM

bsmt_status launched(const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(BSMT_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return BSMT_OK;
}

bsmt_status device(int* dev, int* nsm, int** status) {
    const bsmt_status st = sm_count(dev, nsm);
    return st != BSMT_OK ? st : status_word(*dev, status);
}

// Checks the cache and gives the kernels' form of it.
bsmt_status check_cache(const bsmt_kv_cache* in, bsmt::KvCache* out) {
    if (in == nullptr) return fail(BSMT_ERR_INVALID_ARGUMENT, "cache is NULL");
    if (in->head_dim != 64 && in->head_dim != 128)
        return fail(BSMT_ERR_UNSUPPORTED, "cache head_dim=%d (supported: 64, 128)", in->head_dim);
    if (in->page_size != 16 && in->page_size != 32 && in->page_size != 64 && in->page_size != 128)
        return fail(BSMT_ERR_UNSUPPORTED, "cache page_size=%d (supported: 16, 32, 64, 128)", in->page_size);
    if (in->dtype != BSMT_CACHE_E4M3 && in->dtype != BSMT_CACHE_INT8)
        return fail(BSMT_ERR_UNSUPPORTED, "cache dtype %d", in->dtype);
    if (in->num_layers < 1 || in->num_pages < 1 || in->num_kv_heads < 1 || in->max_seqs < 1 || in->max_pages < 1)
        return fail(BSMT_ERR_INVALID_ARGUMENT, "cache sizes must be positive (layers %d, pages %d, kv heads %d, seqs %d, pages a seq %d)",
                    in->num_layers, in->num_pages, in->num_kv_heads, in->max_seqs, in->max_pages);
    if (in->max_seqs > kMaxSeqs) return fail(BSMT_ERR_UNSUPPORTED, "cache max_seqs=%d above %d", in->max_seqs, kMaxSeqs);
    if (in->num_kv_heads > 65535) return fail(BSMT_ERR_UNSUPPORTED, "cache num_kv_heads=%d above 65535", in->num_kv_heads);
    if (in->num_pages > (1 << 30)) return fail(BSMT_ERR_UNSUPPORTED, "cache num_pages=%d above 2^30", in->num_pages);
    if (int64_t(in->max_pages) * in->page_size > kMaxLen)
        return fail(BSMT_ERR_UNSUPPORTED, "cache: %d pages of %d tokens a sequence, above %lld tokens", in->max_pages,
                    in->page_size, static_cast<long long>(kMaxLen));
    if (!in->k || !in->v || !in->k_scale || !in->v_scale || !in->page_table || !in->seq_lens || !in->ref_counts)
        return fail(BSMT_ERR_INVALID_ARGUMENT, "cache pointers must be non-NULL");
    if (!aligned(in->k, 16) || !aligned(in->v, 16) || !aligned(in->ref_counts, 16))
        return fail(BSMT_ERR_INVALID_ARGUMENT, "cache k, v and ref_counts must be 16-byte aligned");
    if (!aligned(in->k_scale, 4) || !aligned(in->v_scale, 4) || !aligned(in->page_table, 4) || !aligned(in->seq_lens, 4))
        return fail(BSMT_ERR_INVALID_ARGUMENT, "cache scales, page_table and seq_lens must be 4-byte aligned");
    out->k = static_cast<uint8_t*>(in->k);
    out->v = static_cast<uint8_t*>(in->v);
    out->k_scale = in->k_scale;
    out->v_scale = in->v_scale;
    out->page_table = in->page_table;
    out->seq_lens = in->seq_lens;
    out->ref_counts = in->ref_counts;
    out->layers = in->num_layers;
    out->pages = in->num_pages;
    out->heads = in->num_kv_heads;
    out->page = in->page_size;
    out->page_shift = in->page_size == 16 ? 4 : in->page_size == 32 ? 5 : in->page_size == 64 ? 6 : 7;
    out->dim = in->head_dim;
    out->max_seqs = in->max_seqs;
    out->max_pages = in->max_pages;
    out->int8 = in->dtype == BSMT_CACHE_INT8;
    return BSMT_OK;
}

bsmt_status check_layer(const bsmt::KvCache& c, int32_t layer) {
    if (layer < 0 || layer >= c.layers) return fail(BSMT_ERR_INVALID_ARGUMENT, "layer %d outside [0, %d)", layer, c.layers);
    return BSMT_OK;
}

// A list of n int32 on the device.
bsmt_status check_list(const char* name, const int32_t* p, int64_t n, bool optional = false) {
    if (p == nullptr && !optional && n > 0) return fail(BSMT_ERR_INVALID_ARGUMENT, "%s is NULL", name);
    if (!aligned(p, 4)) return fail(BSMT_ERR_INVALID_ARGUMENT, "%s must be 4-byte aligned", name);
    return BSMT_OK;
}

bsmt_status check_count(int64_t n, int64_t T, const int32_t* cu) {
    if (n < 0 || T < 0) return fail(BSMT_ERR_INVALID_ARGUMENT, "negative size (%lld sequences, %lld tokens)",
                                    static_cast<long long>(n), static_cast<long long>(T));
    if (n > (1 << 24) || T > kMaxLen) return fail(BSMT_ERR_UNSUPPORTED, "%lld sequences, %lld tokens", static_cast<long long>(n),
                                                  static_cast<long long>(T));
    if (cu == nullptr && n != T)
        return fail(BSMT_ERR_SHAPE_MISMATCH, "%lld tokens for %lld sequences: cu_seqlens is needed unless there is one each",
                    static_cast<long long>(T), static_cast<long long>(n));
    return BSMT_OK;
}

bsmt_status check_workspace(const void* ws, int64_t have, int64_t need) {
    if (ws == nullptr || !aligned(ws, 256))
        return fail(BSMT_ERR_INVALID_ARGUMENT, "workspace must be non-NULL and 256-byte aligned");
    if (have < need)
        return fail(BSMT_ERR_INVALID_ARGUMENT, "workspace holds %lld bytes, %lld needed", static_cast<long long>(have),
                    static_cast<long long>(need));
    return BSMT_OK;
}

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

#define TRY(x)                             \
    do {                                   \
        const bsmt_status st_ = (x);       \
        if (st_ != BSMT_OK) return st_;    \
    } while (0)

// ------------------------------------------------------------------ rotary
namespace {
template <typename E>
void launch_rotary(const bsmt::RotaryParams& p, int vec, bool interleaved, dim3 grid, cudaStream_t s) {
    constexpr int n = bsmt::kRotaryThreads;
    if (vec == 8) {
        if (interleaved)
            bsmt::rotary_kernel<E, 8, true><<<grid, n, 0, s>>>(p);
        else
            bsmt::rotary_kernel<E, 8, false><<<grid, n, 0, s>>>(p);
    } else {
        if (interleaved)
            bsmt::rotary_kernel<E, 1, true><<<grid, n, 0, s>>>(p);
        else
            bsmt::rotary_kernel<E, 1, false><<<grid, n, 0, s>>>(p);
    }
}
}  // namespace

extern "C" bsmt_status bsmt_rotary_sections(int32_t head_dim, const int32_t* sections, int32_t num_sections, double base,
                                            int32_t per_axis, int32_t interleaved, bsmt_rotary_spec* out) {
    if (out == nullptr || (num_sections > 0 && sections == nullptr))
        return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: sections and out must be non-NULL");
    if (num_sections < 1 || num_sections > 127) return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: %d axes", num_sections);
    if (!(base > 0) || !std::isfinite(base)) return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: base must be finite and > 0");
    int64_t pairs = 0;
    for (int32_t a = 0; a < num_sections; ++a) {
        if (sections[a] < 0) return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: sections[%d] is negative", a);
        pairs += sections[a];
    }
    if (pairs < 1 || pairs > BSMT_MAX_ROTARY_PAIRS || head_dim < 2 * pairs)
        return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: %lld pairs in a head of %d (1 to %d pairs)", static_cast<long long>(pairs), head_dim,
                    BSMT_MAX_ROTARY_PAIRS);
    std::memset(out, 0, sizeof(*out));
    out->head_dim = head_dim;
    out->num_pairs = static_cast<int32_t>(pairs);
    out->num_axes = num_sections;
    out->interleaved = interleaved != 0;
    int32_t i = 0;
    for (int32_t a = 0; a < num_sections; ++a)
        for (int32_t j = 0; j < sections[a]; ++j, ++i) {
            out->inv_freq[i] = per_axis ? std::pow(base, -static_cast<double>(j) / sections[a]) : std::pow(base, -static_cast<double>(i) / pairs);
            out->axis[i] = static_cast<int8_t>(a);
        }
    return ok();
}

extern "C" bsmt_status bsmt_rotary(const bsmt_rotary_spec* spec, int32_t dtype, int64_t B, int64_t T,
                                   const int32_t* positions, const int64_t position_strides[3], int32_t inverse,
                                   const bsmt_rotary_tensor* tensors, int32_t num_tensors, void* stream) {
    if (spec == nullptr || tensors == nullptr || position_strides == nullptr)
        return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: spec, tensors and position_strides must be non-NULL");
    if (dtype != BSMT_BF16 && dtype != BSMT_FP32) return fail(BSMT_ERR_UNSUPPORTED, "rotary dtype %d", dtype);
    if (num_tensors < 1 || num_tensors > 2) return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: %d tensors (1 or 2)", num_tensors);
    if (B < 0 || T < 0) return fail(BSMT_ERR_INVALID_ARGUMENT, "negative size (B=%lld T=%lld)", static_cast<long long>(B), static_cast<long long>(T));
    if (T > kMaxLen || (T > 0 && B > (int64_t(1) << 40) / T)) return fail(BSMT_ERR_UNSUPPORTED, "rotary: B=%lld T=%lld", static_cast<long long>(B), static_cast<long long>(T));
    if (spec->num_pairs < 1 || spec->num_pairs > BSMT_MAX_ROTARY_PAIRS || spec->head_dim < 2 * spec->num_pairs)
        return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: %d pairs in a head of %d (1 to %d pairs)", spec->num_pairs, spec->head_dim,
                    BSMT_MAX_ROTARY_PAIRS);
    if (spec->num_axes < 1 || spec->num_axes > 127) return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: %d axes", spec->num_axes);
    bsmt::RotaryParams p;
    std::memset(&p, 0, sizeof(p));
    for (int i = 0; i < spec->num_pairs; ++i) {
        const double f = spec->inv_freq[i];
        if (!std::isfinite(f)) return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: inv_freq[%d] is not finite", i);
        if (spec->axis[i] < 0 || spec->axis[i] >= spec->num_axes)
            return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: pair %d has axis %d of %d", i, spec->axis[i], spec->num_axes);
        // the fraction of a turn, in 2^-64 turns (whole turns drop out)
        const long double turns = static_cast<long double>(f) / 6.283185307179586476925286766559L;
        const long double part = turns - std::floor(turns);
        p.turn[i] = part < 1.0L ? static_cast<uint64_t>(part * 18446744073709551616.0L) : 0;
        p.axis[i] = spec->axis[i];
    }
    int64_t heads = 0;
    const int64_t size = dtype == BSMT_BF16 ? 2 : 4;
    bool wide = spec->num_pairs % 8 == 0;
    for (int i = 0; i < num_tensors; ++i) {
        const bsmt_rotary_tensor& x = tensors[i];
        if (x.heads < 0) return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: tensor %d has %d heads", i, x.heads);
        if (B * T > 0 && x.heads > 0 && (!x.in || !x.out)) return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: tensor %d is NULL", i);
        if (!aligned(x.in, size) || !aligned(x.out, size)) return fail(BSMT_ERR_INVALID_ARGUMENT, "rotary: tensor %d is misaligned", i);
        wide = wide && aligned(x.in, 16) && aligned(x.out, 16);
        const int64_t extents[3] = {B, x.heads, T};
        for (int j = 0; j < 3; ++j)
            wide = wide && (extents[j] <= 1 || (x.in_strides[j] * size % 16 == 0 && x.out_strides[j] * size % 16 == 0));
        p.x[i] = {x.in, x.out, x.in_strides[0], x.in_strides[1], x.in_strides[2], x.out_strides[0], x.out_strides[1], x.out_strides[2], x.heads};
        heads += x.heads;
    }
    if (heads > 65535) return fail(BSMT_ERR_UNSUPPORTED, "rotary: %lld heads", static_cast<long long>(heads));
    if (B * T == 0 || heads == 0) return ok();
    TRY(check_list("positions", positions, 1));
    int dev = 0, nsm = 0;
    TRY(sm_count(&dev, &nsm));
    p.pos = positions;
    p.pos_axis = position_strides[0];
    p.pos_b = position_strides[1];
    p.pos_t = position_strides[2];
    p.tokens = B * T;
    p.T = static_cast<int32_t>(T);
    p.head_dim = spec->head_dim;
    p.pairs = spec->num_pairs;
    p.heads = static_cast<int32_t>(heads);
    p.inverse = inverse != 0;
    const int vec = wide ? 8 : 1;
    // Where a token's heads lie side by side, a warp takes four of them and reads 1 KB runs; only when the tokens alone
    // fill the machine, since each thread then serves a quarter of the heads with its sines. (30011 tokens of 40 heads:
    // 117 us with one, 110 with four; 48 tokens: 4.1 and 6.2.)
    const int64_t heads_apart = tensors[0].in_strides[1], tokens_apart = tensors[0].in_strides[2];
    p.side = heads >= 16 && heads_apart < tokens_apart && p.tokens * (spec->num_pairs / vec) >= int64_t(nsm) * 4 * bsmt::kRotaryThreads ? 4 : 1;
    const int64_t units = p.tokens * p.side * (spec->num_pairs / vec);
    const int64_t blocks = (units + bsmt::kRotaryThreads - 1) / bsmt::kRotaryThreads;
    if (blocks > 0x7FFFFFFF) return fail(BSMT_ERR_UNSUPPORTED, "rotary: grid too large");
    // A thread's sines serve `chunk` heads: as many as leave some 8 blocks an SM.
    int64_t cuts = std::max<int64_t>(1, std::min<int64_t>(heads, 8 * int64_t(nsm) / blocks));
    p.chunk = static_cast<int32_t>((heads + cuts - 1) / cuts);
    cuts = (heads + p.chunk - 1) / p.chunk;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(cuts));
    if (dtype == BSMT_BF16)
        launch_rotary<__nv_bfloat16>(p, vec, spec->interleaved != 0, grid, static_cast<cudaStream_t>(stream));
    else
        launch_rotary<float>(p, vec, spec->interleaved != 0, grid, static_cast<cudaStream_t>(stream));
    TRY(launched("rotary"));
    return ok();
}

// ------------------------------------------------------------------- cache
namespace {
template <bool INT8>
void launch_write_pages(int nv, unsigned grid, cudaStream_t s, const bsmt::CacheWriteParams& p) {
    if (nv <= 1)
        bsmt::cache_write_pages_kernel<1, INT8><<<grid, 256, 0, s>>>(p);
    else if (nv == 2)
        bsmt::cache_write_pages_kernel<2, INT8><<<grid, 256, 0, s>>>(p);
    else if (nv == 4)
        bsmt::cache_write_pages_kernel<4, INT8><<<grid, 256, 0, s>>>(p);
    else
        bsmt::cache_write_pages_kernel<8, INT8><<<grid, 256, 0, s>>>(p);
}
}  // namespace

extern "C" bsmt_status bsmt_cache_write(const bsmt_kv_cache* cache, int32_t layer, const int32_t* seqs, const int32_t* starts,
                                        int64_t n, const int32_t* cu_seqlens, const void* k, const void* v, int64_t T,
                                        const int64_t k_strides[2], const int64_t v_strides[2], void* stream) {
    bsmt::CacheWriteParams p;
    TRY(check_cache(cache, &p.c));
    TRY(check_layer(p.c, layer));
    TRY(check_count(n, T, cu_seqlens));
    TRY(check_list("seqs", seqs, n));
    TRY(check_list("starts", starts, n));
    TRY(check_list("cu_seqlens", cu_seqlens, 1, true));
    if (n == 0 || T == 0) return ok();
    if (!k || !v || !k_strides || !v_strides) return fail(BSMT_ERR_INVALID_ARGUMENT, "k, v and their strides must be non-NULL");
    for (int i = 0; i < 2; ++i)  // (the stride of one token or head is not used)
        if ((i == 0 ? T : p.c.heads) > 1 && (k_strides[i] % 8 != 0 || v_strides[i] % 8 != 0 || k_strides[i] < 0 || v_strides[i] < 0))
            return fail(BSMT_ERR_INVALID_ARGUMENT, "k and v strides must be multiples of 8 elements");
    if (!aligned(k, 16) || !aligned(v, 16)) return fail(BSMT_ERR_INVALID_ARGUMENT, "k and v must be 16-byte aligned");
    int dev = 0, nsm = 0;
    TRY(device(&dev, &nsm, &p.status));
    p.seqs = seqs;
    p.starts = starts;
    p.cu = cu_seqlens;
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.kt = k_strides[0];
    p.kh = k_strides[1];
    p.vt = v_strides[0];
    p.vh = v_strides[1];
    p.T = T;
    p.n = static_cast<int32_t>(n);
    p.layer = layer;
    p.items = cu_seqlens == nullptr ? n : (T >> p.c.page_shift) + 2 * n;
    // A warp for each page, head and tensor in calls of at most four tokens a sequence on average, else a block for each
    // page and some of the heads: few enough that there are 16 blocks an SM.
    const bool few = T <= 4 * n;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (few) {
        const int64_t blocks = (p.items * 2 * p.c.heads + 7) / 8;
        if (blocks > 0x7FFFFFFF) return fail(BSMT_ERR_UNSUPPORTED, "cache_write: grid too large");
        if (p.c.int8)
            bsmt::cache_write_rows_kernel<true><<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
        else
            bsmt::cache_write_rows_kernel<false><<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
    } else {
        const int64_t heads = 2 * int64_t(p.c.heads);
        p.share = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(heads, p.items * heads / (16 * int64_t(nsm)))));
        const int64_t blocks = p.items * ((heads + p.share - 1) / p.share);
        if (blocks > 0x7FFFFFFF) return fail(BSMT_ERR_UNSUPPORTED, "cache_write: grid too large");
        const unsigned grid = static_cast<unsigned>(blocks);
        const int nv = p.c.page * p.c.dim / 2048;  // vectors of 8 values a thread holds
        if (p.c.int8)
            launch_write_pages<true>(nv, grid, s, p);
        else
            launch_write_pages<false>(nv, grid, s, p);
    }
    TRY(launched("cache_write"));
    return ok();
}

extern "C" bsmt_status bsmt_cache_gather(const bsmt_kv_cache* cache, int32_t layer, const int32_t* seqs, const int32_t* starts,
                                         int64_t n, const int32_t* cu_seqlens, int64_t T, void* k, void* v, void* stream) {
    bsmt::CacheGatherParams p;
    TRY(check_cache(cache, &p.c));
    TRY(check_layer(p.c, layer));
    TRY(check_count(n, T, cu_seqlens));
    TRY(check_list("seqs", seqs, n));
    TRY(check_list("starts", starts, n, true));
    TRY(check_list("cu_seqlens", cu_seqlens, 1, true));
    if (T == 0) return ok();
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16))
        return fail(BSMT_ERR_INVALID_ARGUMENT, "k and v must be non-NULL and 16-byte aligned");
    int dev = 0, nsm = 0;
    TRY(device(&dev, &nsm, &p.status));
    p.seqs = seqs;
    p.starts = starts;
    p.cu = cu_seqlens;
    p.k = static_cast<__nv_bfloat16*>(k);
    p.v = static_cast<__nv_bfloat16*>(v);
    p.T = T;
    p.n = static_cast<int32_t>(n);
    p.layer = layer;
    // Tokens of a block: few enough for 4 blocks an SM, since each finds its tokens' places first.
    p.tokens = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(bsmt::kGatherTokens, T / (4 * int64_t(nsm)))));
    const unsigned grid = static_cast<unsigned>((T + p.tokens - 1) / p.tokens);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.c.int8)
        bsmt::cache_gather_kernel<true><<<grid, 256, 0, s>>>(p);
    else
        bsmt::cache_gather_kernel<false><<<grid, 256, 0, s>>>(p);
    TRY(launched("cache_gather"));
    return ok();
}

// ------------------------------------------------------------------- pages
extern "C" bsmt_status bsmt_cache_workspace_bytes(const bsmt_kv_cache* cache, int64_t n, int64_t* bytes) {
    if (cache == nullptr || bytes == nullptr) return fail(BSMT_ERR_INVALID_ARGUMENT, "cache and bytes must be non-NULL");
    if (cache->num_pages < 1 || n < 0 || n > (1 << 24))
        return fail(BSMT_ERR_INVALID_ARGUMENT, "%d pages, %lld sequences", cache->num_pages, static_cast<long long>(n));
    *bytes = 256 + std::max<int64_t>(3 * round256(int64_t(cache->num_pages) * 4), round256(int64_t(cache->num_pages) * 4) + round256(n * 8));
    return ok();
}

extern "C" bsmt_status bsmt_cache_extend(const bsmt_kv_cache* cache, const int32_t* seqs, const int32_t* counts, int64_t n,
                                         int32_t* starts, void* workspace, int64_t workspace_bytes, void* stream) {
    bsmt::CacheExtendParams p;
    TRY(check_cache(cache, &p.c));
    TRY(check_count(n, n, nullptr));
    TRY(check_list("seqs", seqs, n));
    TRY(check_list("counts", counts, n, true));
    TRY(check_list("starts", starts, n));
    if (n == 0) return ok();
    int64_t need = 0;
    TRY(bsmt_cache_workspace_bytes(cache, n, &need));
    TRY(check_workspace(workspace, workspace_bytes, need));
    int dev = 0, nsm = 0;
    TRY(device(&dev, &nsm, &p.status));
    p.seqs = seqs;
    p.counts = counts;
    p.starts = starts;
    p.list = static_cast<int32_t*>(workspace);
    p.n = static_cast<int32_t>(n);
    const int bitmap = (p.c.max_seqs + 31) / 32 * 4;
    bsmt::cache_extend_kernel<<<1, bsmt::kPlanThreads, bitmap, static_cast<cudaStream_t>(stream)>>>(p);
    TRY(launched("cache_extend"));
    return ok();
}

extern "C" bsmt_status bsmt_cache_fork(const bsmt_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t n,
                                       void* workspace, int64_t workspace_bytes, void* stream) {
    bsmt::CacheForkParams p;
    TRY(check_cache(cache, &p.c));
    TRY(check_count(n, n, nullptr));
    TRY(check_list("src", src, n));
    TRY(check_list("dst", dst, n));
    if (n == 0) return ok();
    int64_t need = 0;
    TRY(bsmt_cache_workspace_bytes(cache, n, &need));
    TRY(check_workspace(workspace, workspace_bytes, need));
    int dev = 0, nsm = 0;
    TRY(device(&dev, &nsm, &p.status));
    p.src = src;
    p.dst = dst;
    p.list = static_cast<int32_t*>(workspace);
    p.jobs = reinterpret_cast<int2*>(static_cast<char*>(workspace) + round256(int64_t(p.c.pages) * 4));
    p.n = static_cast<int32_t>(n);
    // Blocks of one fork: a warp for each head of k and v of a layer, and some 8 blocks an SM in all.
    const int64_t spans = int64_t(p.c.layers) * 2 * p.c.heads;
    p.blocks = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>((spans + 7) / 8, std::max<int64_t>(2, 8 * int64_t(nsm) / n))));
    const int bitmap = (p.c.max_seqs + 31) / 32 * 4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    bsmt::cache_fork_plan_kernel<<<1, bsmt::kPlanThreads, bitmap, s>>>(p);
    TRY(launched("cache_fork plan"));
    bsmt::cache_fork_kernel<<<static_cast<unsigned>(n * p.blocks), 256, 0, s>>>(p);
    TRY(launched("cache_fork"));
    return ok();
}

extern "C" bsmt_status bsmt_cache_free(const bsmt_kv_cache* cache, const int32_t* seqs, int64_t n, void* stream) {
    bsmt::KvCache c;
    TRY(check_cache(cache, &c));
    TRY(check_count(n, n, nullptr));
    TRY(check_list("seqs", seqs, n));
    if (n == 0) return ok();
    int dev = 0, nsm = 0;
    int* status = nullptr;
    TRY(device(&dev, &nsm, &status));
    bsmt::cache_free_kernel<<<static_cast<unsigned>(n), 256, 0, static_cast<cudaStream_t>(stream)>>>(c, seqs, status);
    TRY(launched("cache_free"));
    return ok();
}

extern "C" bsmt_status bsmt_cache_compact(const bsmt_kv_cache* cache, int32_t* live, void* workspace, int64_t workspace_bytes,
                                          void* stream) {
    bsmt::CacheCompactParams p;
    TRY(check_cache(cache, &p.c));
    TRY(check_list("live", live, 1));
    int64_t need = 0;
    TRY(bsmt_cache_workspace_bytes(cache, 0, &need));
    TRY(check_workspace(workspace, workspace_bytes, need));
    int dev = 0, nsm = 0;
    TRY(device(&dev, &nsm, &p.status));
    const int64_t list = round256(int64_t(p.c.pages) * 4) / 4;
    p.live = live;
    p.header = static_cast<int32_t*>(workspace);
    p.holes = p.header + 64;
    p.movers = p.holes + list;
    p.to = p.movers + list;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    bsmt::cache_compact_plan_kernel<<<1, bsmt::kPlanThreads, 0, s>>>(p);
    TRY(launched("cache_compact plan"));
    {
        std::lock_guard<std::mutex> lk(g_set_mu);
        if (!g_compact_set[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(bsmt::cache_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bsmt::kCompactSmem);
            if (e != cudaSuccess) return fail(BSMT_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            g_compact_set[dev] = true;
        }
    }
    bsmt::cache_compact_kernel<<<3 * nsm, 128, bsmt::kCompactSmem, s>>>(p);
    TRY(launched("cache_compact"));
    return ok();
}

// --------------------------------------------------------------- attention
namespace {


// O, the maxima and sums of two parts for each block, and the blocks' heads.
int64_t paged_ws_bytes(int64_t D) {
    return int64_t(kMaxPartRows) * 2 * (D + 4) * 4 + round256(int64_t(kMaxPartBlocks) * 32);
}

template <int D, bool INT8, int NT, int MODS>
bsmt_status launch_paged(int dev, int nsm, bsmt::PagedParams p, const bsmt::MaskDnf& dnf, cudaStream_t s) {
    auto kern = bsmt::paged_attention_kernel<D, INT8, NT, MODS>;
    constexpr int smem = bsmt::PagedShape<D, NT>::kSmem;
    {
        std::lock_guard<std::mutex> lk(g_set_mu);
        bool& set = g_paged_set[dev][(D == 128 ? 18 : 0) + (INT8 ? 9 : 0) + (NT / 2) * 3 + MODS];
        if (!set) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return fail(BSMT_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            set = true;
        }
    }
    const int blocks = std::min({bsmt::PagedShape<D, NT>::kBlocks * nsm, kMaxPartBlocks, kMaxPartRows / (8 * NT)});
    // the pools as rows of D codes; a copy takes the rows of a tile that lie in one page
    const int64_t rows = int64_t(p.c.layers) * p.c.pages * p.c.heads * p.c.page;
    CUtensorMap k_map, v_map;
    TRY(encode_rows(&k_map, p.c.k, rows, D, std::min(p.c.page, bsmt::kTileTokens)));
    TRY(encode_rows(&v_map, p.c.v, rows, D, std::min(p.c.page, bsmt::kTileTokens)));
    // Each kernel is set up while the one before it in the stream runs, and waits for that one's end on the device
    // before it reads anything.
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * bsmt::PagedShape<D, NT>::kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    (void)cudaLaunchKernelEx(&cfg, kern, p, dnf, k_map, v_map);
    TRY(launched("paged_attention"));  // (reads the error and clears it, so that the next call does not find it)
    cfg.gridDim = dim3(blocks, 2 * NT);
    cfg.blockDim = dim3(32 * bsmt::kCombineWarps);
    cfg.dynamicSmemBytes = 0;
    (void)cudaLaunchKernelEx(&cfg, bsmt::paged_combine_kernel<D, 8 * NT>, p);
    TRY(launched("paged_attention combine"));
    return BSMT_OK;
}

template <int D, bool INT8, int NT>
bsmt_status launch_paged_mods(int mods, int dev, int nsm, const bsmt::PagedParams& p, const bsmt::MaskDnf& dnf, cudaStream_t s) {
    if (mods == 0) return launch_paged<D, INT8, NT, 0>(dev, nsm, p, dnf, s);
    return mods == 1 ? launch_paged<D, INT8, NT, 1>(dev, nsm, p, dnf, s) : launch_paged<D, INT8, NT, 2>(dev, nsm, p, dnf, s);
}

template <int D, bool INT8>
bsmt_status launch_paged_kind(int nt, int mods, int dev, int nsm, const bsmt::PagedParams& p, const bsmt::MaskDnf& dnf, cudaStream_t s) {
    if (nt == 1) return launch_paged_mods<D, INT8, 1>(mods, dev, nsm, p, dnf, s);
    if (nt == 2 || D == 128) return launch_paged_mods<D, INT8, 2>(mods, dev, nsm, p, dnf, s);
    return launch_paged_mods<D, INT8, D == 64 ? 4 : 2>(mods, dev, nsm, p, dnf, s);
}

}  // namespace

extern "C" bsmt_status bsmt_paged_attention_workspace_bytes(int64_t D, int64_t* bytes) {
    if (bytes == nullptr) return fail(BSMT_ERR_INVALID_ARGUMENT, "bytes is NULL");
    if (D != 64 && D != 128) return fail(BSMT_ERR_UNSUPPORTED, "head dim D=%lld (supported: 64, 128)", static_cast<long long>(D));
    *bytes = paged_ws_bytes(D);
    return ok();
}

extern "C" bsmt_status bsmt_paged_attention(const void* q, int64_t T, int64_t Hq, const bsmt_kv_cache* cache, int32_t layer,
                                            const int32_t* seqs, int64_t n, const int32_t* cu_seqlens_q,
                                            const bsmt_mask_spec* mask_spec, const bsmt_score_spec* score, float scale,
                                            int32_t enable_gqa, void* out, float* lse, void* workspace,
                                            int64_t workspace_bytes, void* stream) {
    bsmt::PagedParams p;
    std::memset(&p, 0, sizeof(p));
    TRY(check_cache(cache, &p.c));
    TRY(check_layer(p.c, layer));
    TRY(check_count(n, T, cu_seqlens_q));
    TRY(check_list("seqs", seqs, n));
    TRY(check_list("cu_seqlens_q", cu_seqlens_q, 1, true));
    if (Hq < 1 || Hq > 65535 || Hq % p.c.heads != 0)
        return fail(BSMT_ERR_SHAPE_MISMATCH, "Hq=%lld is not a multiple of the cache's %d kv heads", static_cast<long long>(Hq), p.c.heads);
    if (Hq != p.c.heads && !enable_gqa)
        return fail(BSMT_ERR_SHAPE_MISMATCH, "Hq=%lld != Hkv=%d requires enable_gqa", static_cast<long long>(Hq), p.c.heads);
    if (T > 0 && (!q || !out || !lse)) return fail(BSMT_ERR_INVALID_ARGUMENT, "q, out and lse must be non-NULL");
    if (!aligned(q, 16) || !aligned(out, 16)) return fail(BSMT_ERR_INVALID_ARGUMENT, "q and out must be 16-byte aligned");
    if (!aligned(lse, 4)) return fail(BSMT_ERR_INVALID_ARGUMENT, "lse must be 4-byte aligned");
    if (std::isnan(scale) || std::isinf(scale)) return fail(BSMT_ERR_INVALID_ARGUMENT, "scale must be finite");
    if (scale <= 0.f) scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(p.c.dim)));
    if (mask_spec != nullptr)
        for (int i = 0; i < mask_spec->num_nodes && i < BSMT_MAX_MASK_NODES; ++i)
            if (mask_spec->nodes[i].kind == BSMT_MASK_DOCUMENT)
                return fail(BSMT_ERR_UNSUPPORTED, "paged attention: a cache's sequence is one document; DOCUMENT masks are not taken");
    bsmt::MaskDnf dnf;
    TRY(build_dnf(mask_spec, 1, &dnf));
    ScoreArgs sa;
    TRY(score_args(score, Hq, &sa));
    if (int64_t(p.c.layers) * p.c.pages * p.c.heads * p.c.page > kMaxLen)
        return fail(BSMT_ERR_UNSUPPORTED, "paged attention: a pool of %d layers, %d pages and %d heads has more than %lld rows",
                    p.c.layers, p.c.pages, p.c.heads, static_cast<long long>(kMaxLen));
    if (T == 0) return ok();
    TRY(check_workspace(workspace, workspace_bytes, paged_ws_bytes(p.c.dim)));
    int dev = 0, nsm = 0;
    TRY(device(&dev, &nsm, &p.status));
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.seqs = seqs;
    p.cu = cu_seqlens_q;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.part_o = static_cast<float*>(workspace);
    p.part_m = p.part_o + int64_t(kMaxPartRows) * 2 * p.c.dim;
    p.heads_of_parts = reinterpret_cast<int32_t*>(p.part_m + int64_t(kMaxPartRows) * 2 * 4);
    p.slopes = sa.slopes;
    p.T = T;
    p.n = static_cast<int32_t>(n);
    p.layer = layer;
    p.Hq = static_cast<int32_t>(Hq);
    p.group = static_cast<int32_t>(Hq / p.c.heads);
    p.min_share = 8;  // two tiles for each warp of a block
    p.scale = scale;
    p.cap = sa.cap;
    p.cap_inv = static_cast<float>(std::min((sa.cap <= 64.f ? 2.0 * 1.4426950408889634 : 1.0) / sa.cap, static_cast<double>(FLT_MAX)));
    // the modes of the score program: none, soft-cap, ALiBi, soft-cap then ALiBi, ALiBi then soft-cap
    p.softcap = sa.mode == 1 || sa.mode == 3 || sa.mode == 4;
    p.alibi_first = sa.mode == 4;
    p.alibi_h0 = sa.alibi_h0;
    p.alibi_heads = sa.alibi_heads;
    // Row tiles of 8 or 16, or, at D = 64, 32: the smallest that holds an average sequence's rows, so that its keys are
    // read once. (32 rows of 24 sequences up to 64k: 32 a tile 377 us and 16 a tile 438 us at D = 64; at D = 128 O spills
    // with 32, which took 1.14 times as long as two tiles of 16.)
    const int64_t rows = (T * p.group + std::max<int64_t>(n, 1) - 1) / std::max<int64_t>(n, 1);
    const int nt = rows <= 8 ? 1 : rows <= 16 || p.c.dim == 128 ? 2 : 4;
    const int mods = sa.mode <= 1 ? sa.mode : 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    bsmt_status st;
    if (p.c.dim == 128)
        st = p.c.int8 ? launch_paged_kind<128, true>(nt, mods, dev, nsm, p, dnf, s) : launch_paged_kind<128, false>(nt, mods, dev, nsm, p, dnf, s);
    else
        st = p.c.int8 ? launch_paged_kind<64, true>(nt, mods, dev, nsm, p, dnf, s) : launch_paged_kind<64, false>(nt, mods, dev, nsm, p, dnf, s);
    if (st != BSMT_OK) return st;
    return ok();
}
