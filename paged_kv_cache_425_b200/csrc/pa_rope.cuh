// Rotary positions with several axes, fused with the cache write.
//
// Pair i of a head, (x, y) = elements (i, i + P) or (2i, 2i + 1) of its first
// 2P elements, turns by the angle positions[axis(i)][t] * inv_freq[i]:
//   x' = x cos - y sin,  y' = y cos + x sin.
// The angle is held as a 64-bit fraction of a turn: the position times the
// fraction of one step (pa_rope_init), modulo 2^64.  The multiplication wraps
// exactly where whole turns drop out, so a far position needs no range
// reduction and adds only the step's own rounding (under 2^-63 of a turn, 2^-32
// at position 2^31, for frequencies up to 1); cos and sin come from sincospif
// of the top 32 bits, in f32, and each output is rounded once.
//
// Memory bound (every q, k, v element is read once and written once; the
// angles are shared by all heads of a token).  One CTA per token: its threads
// put their 16-byte loads in flight, some of them compute the token's P angles
// meanwhile, and after one barrier each thread turns what it loaded.  8192
// tokens of 32 + 8 + 8 heads of 128 (201 MB) take 35.4 us, 0.87 of the measured
// copy bandwidth; 64 tokens 2.8 us, a launch.  128 threads with three units
// each were the fastest of six shapes (256 x 2: 49 us, 64 x 6: 36 us, 128 x 6:
// 41 us); streaming or uncached loads and a tighter register limit gained
// nothing.
#pragma once

#include "pa_kernels.cuh"

namespace pa {

constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 3;  // units in flight per thread

struct RopeArgs {
    uint4 *q_out;
    const uint4 *q, *k, *v;
    uint4 *key_cache, *value_cache;
    const int64_t *slots;
    const int32_t *positions;
    long long q_stride, k_stride, v_stride;  // 16-byte vectors per token
    long long num_slots;
    int num_tokens, num_q_heads, num_kv_heads;
    pa_rope rope;
};

template <typename T>
__device__ __forceinline__ void rope_turn(uint32_t &x, uint32_t &y, const float2 &cs0,
                                          const float2 &cs1) {
    // two pairs: the low halves turn by cs0, the high halves by cs1
    const float2 a = widen2(x, T()), b = widen2(y, T());
    x = Mma<T>::pack(a.x * cs0.x - b.x * cs0.y, a.y * cs1.x - b.y * cs1.y);
    y = Mma<T>::pack(b.x * cs0.x + a.x * cs0.y, b.y * cs1.x + a.y * cs1.y);
}

template <typename T>
__device__ __forceinline__ void rope_turn_next(uint32_t &x, const float2 &cs) {
    const float2 a = widen2(x, T());  // one pair of neighbours
    x = Mma<T>::pack(a.x * cs.x - a.y * cs.y, a.y * cs.x + a.x * cs.y);
}

// A unit is two 16-byte vectors of one head: the two halves of eight pairs
// (elements i and i + P), or 16 elements side by side.
template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int VPR = D / 8, UNITS = VPR / 2;
    __shared__ __align__(16) float2 s_cs[PA_ROPE_MAX_PAIRS];  // cos, sin
    const int t = blockIdx.x;
    const int pairs = a.rope.num_pairs, half8 = pairs / 8;
    const bool next = a.rope.interleaved;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int heads = a.num_q_heads + 2 * a.num_kv_heads;
    const int units = heads * UNITS;
    long long slot = a.slots[t];  // needed for the stores only

    bool ready = false;
    for (int w0 = threadIdx.x; w0 < units || !ready; w0 += kRopeThreads * kRopeUnroll) {
        uint4 x[kRopeUnroll], y[kRopeUnroll];
        int head[kRopeUnroll], c0[kRopeUnroll], c1[kRopeUnroll];
        bool turn[kRopeUnroll];
#pragma unroll
        for (int r = 0; r < kRopeUnroll; ++r) {
            const int w = w0 + r * kRopeThreads;
            const int h = w / UNITS, u = w % UNITS;
            const bool halves = !next && u < half8;
            c0[r] = halves ? u : 2 * u;
            c1[r] = halves ? u + half8 : 2 * u + 1;
            const int hk = h - a.num_q_heads, hv = hk - a.num_kv_heads;
            turn[r] = hv < 0 && c0[r] < 2 * half8;
            head[r] = h;
            if (w >= units) continue;
            const uint4 *src = hk < 0   ? a.q + (size_t)t * a.q_stride + (size_t)h * VPR
                               : hv < 0 ? a.k + (size_t)t * a.k_stride + (size_t)hk * VPR
                                        : a.v + (size_t)t * a.v_stride + (size_t)hv * VPR;
            x[r] = src[c0[r]];
            y[r] = src[c1[r]];
        }
        if (!ready) {
            if (threadIdx.x < pairs) {
                const int i = threadIdx.x;
                const int32_t p = a.positions[(size_t)a.rope.axis[i] * a.num_tokens + t];
                const uint64_t phase = (uint64_t)(int64_t)p * a.rope.turns[i];
                // top 32 bits, signed: half turns in [-1, 1)
                const float turns = (float)(int32_t)(phase >> 32) * 0x1p-31f;
                float sn, cn;
                sincospif(turns, &sn, &cn);
                s_cs[i] = make_float2(cn, sn);
            }
            __syncthreads();
            ready = true;
            if (slot >= a.num_slots) {
                if (threadIdx.x == 0) flag_error(PA_DEVERR_SLOT);
                slot = -1;
            }
        }
        const size_t cache_row =
            slot < 0 ? 0 : (size_t)(slot / kBlock) * a.num_kv_heads * kBlock + slot % kBlock;
#pragma unroll
        for (int r = 0; r < kRopeUnroll; ++r) {
            const int hk = head[r] - a.num_q_heads, hv = hk - a.num_kv_heads;
            if (w0 + r * kRopeThreads >= units || (hk >= 0 && slot < 0)) continue;
            if (turn[r]) {
                uint32_t *xs = reinterpret_cast<uint32_t *>(&x[r]);
                uint32_t *ys = reinterpret_cast<uint32_t *>(&y[r]);
                if (next) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        rope_turn_next<T>(xs[e], s_cs[4 * c0[r] + e]);
                        if (c1[r] < 2 * half8) rope_turn_next<T>(ys[e], s_cs[4 * c1[r] + e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        rope_turn<T>(xs[e], ys[e], s_cs[8 * c0[r] + 2 * e], s_cs[8 * c0[r] + 2 * e + 1]);
                }
            }
            uint4 *dst = hk < 0   ? a.q_out + ((size_t)t * a.num_q_heads + head[r]) * VPR
                         : hv < 0 ? a.key_cache + (cache_row + (size_t)hk * kBlock) * VPR
                                  : a.value_cache + (cache_row + (size_t)hv * kBlock) * VPR;
            dst[c0[r]] = x[r];
            dst[c1[r]] = y[r];
        }
    }
}

}  // namespace pa
