// Rotary positions with several axes, and their gradient.
//
// A head's first 2 * num_pairs elements form pairs (a, b): (x[i], x[i + num_pairs])
// or, interleaved, (x[2i], x[2i + 1]). Pair i turns by t_i = pos[axis_i] * inv_freq_i:
//   a' = a cos t - b sin t,  b' = a sin t + b cos t.
// The map is orthogonal, so the gradient is the turn by -t. Elements behind the
// pairs pass through.
//
// The angle: inv_freq / 2pi is held as a 64-bit fraction of a turn. The product
// with a 32-bit position, taken modulo 2^64, is the exact fraction of the turn
// left after whole turns, so a far position costs no accuracy (the fraction is cut
// off below 2^-64 turns, which times 2^31 positions is 2^-33 turns; an inv_freq of
// whole turns keeps as many bits less of it) and no 64-bit floating point. Its top 32 bits give the angle to sincospif, in half turns.
//
// Bound by HBM: x is read once and written once. A thread keeps the sines of
// its eight pairs of one token in registers and goes over heads of q and k with
// them, one head's 32 bytes in and out at a time: more blocks on an SM hide the
// reads better than more heads in one thread (two blocks with four heads each
// 159 us, four with one 117 us, for 30011 tokens of 40 heads of 128).
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "bsmt_serving.h"
#include "kv_cache.cuh"

namespace bsmt {

constexpr int kRotaryThreads = 256;

struct RotaryTensor {
    const void* in;
    void* out;
    int64_t ib, ih, it, ob, oh, ot;  // element strides: batch, head, token
    int32_t heads;
};

struct RotaryParams {
    uint64_t turn[BSMT_MAX_ROTARY_PAIRS];  // inv_freq / 2pi as a fraction of 2^64
    int8_t axis[BSMT_MAX_ROTARY_PAIRS];
    RotaryTensor x[2];
    const int32_t* pos;
    int64_t pos_axis, pos_b, pos_t;
    int64_t tokens;  // B * T
    int32_t T, head_dim, pairs, heads, chunk, side, inverse;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

// Row (b, h, t) of the call's head h: q's heads, then k's.
template <typename E>
__device__ __forceinline__ E* rotary_row(const RotaryParams& p, int h, int64_t b, int64_t t, bool out) {
    const bool second = h >= p.x[0].heads;
    const RotaryTensor& x = second ? p.x[1] : p.x[0];
    const int hh = second ? h - p.x[0].heads : h;
    return out ? static_cast<E*>(x.out) + b * x.ob + hh * x.oh + t * x.ot
               : static_cast<E*>(const_cast<void*>(x.in)) + b * x.ib + hh * x.ih + t * x.it;
}

// VEC: pairs of one thread, 8 where every row is 16-byte aligned and the pair
// count a multiple of 8, else 1. A load is at most 16 bytes.
template <typename E, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads, 4) rotary_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ uint64_t s_turn[BSMT_MAX_ROTARY_PAIRS];
    __shared__ int8_t s_axis[BSMT_MAX_ROTARY_PAIRS];
    for (int i = threadIdx.x; i < p.pairs; i += kRotaryThreads) {
        s_turn[i] = p.turn[i];
        s_axis[i] = p.axis[i];
    }
    __syncthreads();
    constexpr int L = 16 / sizeof(E) < VEC ? 16 / sizeof(E) : VEC;  // elements of one load
    constexpr int NL = VEC / L;
    const int groups = p.pairs / VEC;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kRotaryThreads + threadIdx.x;
    const int64_t lane_unit = unit / groups;  // (token, which of the heads that go side by side)
    const int64_t token = lane_unit / p.side;
    if (token >= p.tokens) return;
    const int first = static_cast<int>(unit - lane_unit * groups) * VEC;
    const int side = static_cast<int>(lane_unit - token * p.side);
    const int64_t b = token / p.T, t = token - b * p.T;

    float cs[VEC], sn[VEC];
    int last_axis = -1;
    int64_t pos = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int axis = s_axis[first + i];
        if (axis != last_axis) {
            pos = __ldg(p.pos + axis * p.pos_axis + b * p.pos_b + t * p.pos_t);
            last_axis = axis;
        }
        const uint64_t turn = static_cast<uint64_t>(pos) * s_turn[first + i];
        const float half = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
        sincospif(half, &sn[i], &cs[i]);
        if (p.inverse) sn[i] = -sn[i];
    }

    const int h1 = min(p.heads, static_cast<int>(blockIdx.y + 1) * p.chunk);
    const int at_a = INTERLEAVED ? 2 * first : first;
    const int at_b = INTERLEAVED ? 2 * first + VEC : p.pairs + first;  // (interleaved: the second half of 2 * VEC)
    for (int h = blockIdx.y * p.chunk + side; h < h1; h += p.side) {
        const E* in = rotary_row<E>(p, h, b, t, false);
        E* out = rotary_row<E>(p, h, b, t, true);
        Pack<E, L> va[NL], vb[NL];
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            va[j] = *reinterpret_cast<const Pack<E, L>*>(in + at_a + j * L);
            vb[j] = *reinterpret_cast<const Pack<E, L>*>(in + at_b + j * L);
        }
        Pack<E, L> ra[NL], rb[NL];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            // element e of the thread's 2 * VEC lies in va for e < VEC, else in vb
            const int ea = INTERLEAVED ? 2 * i : i, eb = INTERLEAVED ? 2 * i + 1 : VEC + i;
            const float a = to_f32(ea < VEC ? va[ea / L % NL].v[ea % L] : vb[(ea - VEC) / L % NL].v[ea % L]);
            const float c = to_f32(eb < VEC ? va[eb / L % NL].v[eb % L] : vb[(eb - VEC) / L % NL].v[eb % L]);
            E ya, yb;
            from_f32(fmaf(a, cs[i], -(c * sn[i])), ya);
            from_f32(fmaf(a, sn[i], c * cs[i]), yb);
            (ea < VEC ? ra[ea / L % NL].v[ea % L] : rb[(ea - VEC) / L % NL].v[ea % L]) = ya;
            (eb < VEC ? ra[eb / L % NL].v[eb % L] : rb[(eb - VEC) / L % NL].v[eb % L]) = yb;
        }
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            *reinterpret_cast<Pack<E, L>*>(out + at_a + j * L) = ra[j];
            *reinterpret_cast<Pack<E, L>*>(out + at_b + j * L) = rb[j];
        }
        if (2 * p.pairs < p.head_dim)
            for (int e = 2 * p.pairs + first / VEC; e < p.head_dim; e += groups) out[e] = in[e];
    }
}

}  // namespace bsmt
