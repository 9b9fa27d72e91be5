// Decode attention over a sliding window and the first tokens (sinks) of a
// paged context, for one new token per sequence or a short chunk of them.
//
// The query at position p sees token j when j <= p and (p - j < window or
// j < num_sinks).  Over the n query tokens of one sequence (n = 1: decode) the
// visible tokens are the sinks [0, num_sinks) and the window [lo, L) with
// lo = max(0, L - n - window + 1).  Only the blocks that hold such a token are
// read: they are numbered 0 .. nv - 1 (the sink blocks, then the window's), and
// everything below works on that list, so the cost does not depend on L and the
// table entries in between may be empty.
//
// Memory bound: a visible token costs 4 * head_dim bytes per kv head and
// 4 * rows * head_dim flops.  So the kernel has the shape of decode_mma_kernel:
// many resident warps, each with its own small TMA pipeline, and the rows
// (query heads of the group, times the tokens of a chunk) as the N side of one
// mma.sync tile against the 16 tokens of a block.
#pragma once

#include "pa_kernels.cuh"

namespace pa {

struct WindowArgs {
    DecodeArgs d;                // num_parts, part_blocks: of the visible blocks
    const int32_t *query_start;  // chunks only: [S + 1]
    int num_q_tokens;            // rows of q / out
    int max_query_len;           // 1 for decode
    int tile_tokens;             // query tokens that share one list of visible blocks
    int window;                  // >= 1
    int num_sinks;               // >= 0
};

// Query tokens and visible blocks of one sequence.
struct WindowSeq {
    int q0, n, L;  // first query token, query tokens, context length
    int lo;        // first token inside any row's window
    int nsb;       // sink blocks in front of the window's blocks
    int skip;      // blocks between them, with no visible token
    int nv;        // visible blocks
    // logical block of visible block v
    __device__ __forceinline__ int block(int v) const { return v < nsb ? v : v + skip; }
};

__device__ __forceinline__ void window_blocks(WindowSeq &w, int first_pos, int end, int window,
                                              int num_sinks) {
    // visible blocks of queries at first_pos .. end - 1
    w.lo = max(0, first_pos - window + 1);
    const int b0 = w.lo / kBlock;
    w.nsb = min((min(num_sinks, end) + kBlock - 1) / kBlock, b0);
    w.skip = b0 - w.nsb;
    w.nv = (end + kBlock - 1) / kBlock - w.skip;
}

// False when the sequence's query rows lie outside q / out (reported).
template <bool CHUNK>
__device__ __forceinline__ bool window_seq(const WindowArgs &a, int s, bool report, WindowSeq &w) {
    if constexpr (!CHUNK) {
        w.q0 = s;
        w.L = clamp_context(a.d, s, report);
        w.n = w.L > 0 ? 1 : 0;
    } else {
        w.q0 = a.query_start[s];
        w.n = a.query_start[s + 1] - w.q0;
        w.L = a.d.context_lens[s];
        const int cap = a.d.max_blocks_per_seq * kBlock;
        if (w.q0 < 0 || w.q0 > a.num_q_tokens || w.n > a.num_q_tokens - w.q0) {
            if (report) flag_error(PA_DEVERR_CONTEXT_LEN);
            return false;
        }
        if (w.L < 0 || w.L > cap || w.n < 0 || w.n > w.L) {
            if (report) flag_error(PA_DEVERR_CONTEXT_LEN);
            w.L = min(max(w.L, 0), cap);
            w.n = min(max(w.n, 0), w.L);
        }
        if (w.n > a.max_query_len) {
            if (report) flag_error(PA_DEVERR_CONTEXT_LEN);
            return false;
        }
    }
    window_blocks(w, w.L - w.n, w.L, a.window, a.num_sinks);
    return true;
}

// NT 8-row column tiles: rows of a kv head (tokens x group) <= 8 * NT.
template <typename T, int D, int NW, int STAGES, int NT, int PB, bool CHUNK>
__global__ void __launch_bounds__(NW * 32, NT == 1 ? PA_DECODE_MIN_CTAS : 3)
    decode_window_kernel(const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv, const WindowArgs wa) {
    using Pipe = WarpPipe<D, STAGES>;
    const DecodeArgs &a = wa.d;
    constexpr int KS = D / 16;     // 16-wide steps of the head dim
    constexpr int RMAX = 8 * NT;   // rows this build handles
    static_assert(RMAX * D * 4 <= STAGES * Pipe::kStage, "combine scratch fits in a warp ring");
    static_assert(PB <= 32 * NW, "a lane holds one block id");
    extern __shared__ uint8_t dyn_smem[];
    __shared__ __align__(8) uint64_t bars[NW][STAGES];
    __shared__ float s_m[NW][RMAX], s_l[NW][RMAX];

    const int part = blockIdx.y, kvh = blockIdx.x % a.num_kv_heads,
              s = blockIdx.x / a.num_kv_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.num_q_heads / a.num_kv_heads;
    pdl_launch_dependents();
    pdl_wait_prior();
    WindowSeq w;
    if (!window_seq<CHUNK>(wa, s, part == 0 && kvh == 0 && threadIdx.x == 0, w)) return;
    const int rows = CHUNK ? w.n * G : G;
    const int nparts = w.n > 0 ? (w.nv + PB - 1) / PB : 0;
    if (part >= (nparts > 0 ? nparts : 1)) return;
    uint16_t *out = reinterpret_cast<uint16_t *>(a.out);
    // row r of the sequence -> row of q / out
    auto q_row = [&](int r) {
        return CHUNK ? (size_t)(w.q0 + r / G) * a.num_q_heads + (size_t)kvh * G + r % G
                     : (size_t)s * a.num_q_heads + (size_t)kvh * G + r;
    };
    if (w.n == 0) {
        if (!CHUNK)
            for (int i = threadIdx.x; i < G * D; i += NW * 32) out[q_row(0) * D + i] = 0;
        return;
    }
    const int v_begin = part * PB;
    const int nv_local = min(PB, w.nv - v_begin);
    const int nk = warp_block_count(nv_local, warp, NW);

    Pipe pipe;
    pipe.ring = align_smem_1024(dyn_smem) + warp * STAGES * Pipe::kStage;
    pipe.bar = bars[warp];
    pipe.tmk = &tmk;
    pipe.tmv = &tmv;
    pipe.policy = l2_policy_evict_first();
    pipe.kvh = kvh;
    pipe.num_kv_heads = a.num_kv_heads;
    pipe.lane = lane;
    pipe.my_phys = -1;
    if (lane < nk) {
        const int phys =
            a.block_tables[(size_t)s * a.max_blocks_per_seq + w.block(v_begin + warp + lane * NW)];
        if (phys < 0 || phys >= a.num_blocks)
            flag_error(PA_DEVERR_BLOCK_ID);
        else
            pipe.my_phys = phys;
    }
    if (lane == 0) {
        for (int i = 0; i < STAGES; ++i) mbar_init(&bars[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    int issued = nk < STAGES ? nk : STAGES;
    // the new token's write (pa_decode_append_window) goes before the load of
    // its block, which is the last visible one: as in decode_mma_kernel
    int k_app = -1;
    if (!CHUNK && a.k_new != nullptr && a.context_lens[s] == w.L) {
        const int li = w.nv - 1 - v_begin;
        if (li >= 0 && li < nv_local && li % NW == warp) k_app = li / NW;
    }
    if (k_app >= 0 && k_app < issued) append_new_token<D>(a, s, kvh, w.L, lane);
    for (int k = 0; k < issued; ++k) pipe.issue(k);
    if (k_app >= issued) append_new_token<D>(a, s, kvh, w.L, lane);

    const int g = lane >> 2, c = lane & 3;
    // B operand of S^T = K Q^T: lane holds Q[row = 8 nt + g][16 kk + 2c .. +1] and [.. + 8 ..].
    uint32_t qf[NT][KS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
        const uint16_t *qrow = reinterpret_cast<const uint16_t *>(a.q) + (r < rows ? q_row(r) : 0) * D;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            qf[nt][kk][0] = r < rows ? *reinterpret_cast<const uint32_t *>(qrow + 16 * kk + 2 * c) : 0u;
            qf[nt][kk][1] =
                r < rows ? *reinterpret_cast<const uint32_t *>(qrow + 16 * kk + 8 + 2 * c) : 0u;
        }
    }
    // position of rows 8 nt + 2c + j (chunks only; one position otherwise)
    int pos[NT][2];
    if constexpr (CHUNK) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) pos[nt][j] = w.L - w.n + min(nt * 8 + 2 * c + j, rows - 1) / G;
    }
    // Running softmax state per (tile nt, row 2c + j), and O^T accumulators:
    // acc[nt][j] holds d = 16 j + g (+8), rows 8 nt + 2c (+1).
    float mrow[NT][2], lrow[NT][2], acc[NT][KS][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        mrow[nt][0] = mrow[nt][1] = -INFINITY;
        lrow[nt][0] = lrow[nt][1] = 0.f;
#pragma unroll
        for (int j = 0; j < KS; ++j) acc[nt][j][0] = acc[nt][j][1] = acc[nt][j][2] = acc[nt][j][3] = 0.f;
    }
    const int ka_row = (lane & 7) + ((lane >> 3) & 1) * 8, ka_half = lane >> 4;
    const int va_row = (lane & 7) + 8 * (lane >> 4), va_half = (lane >> 3) & 1;

    bool dead = false;
    int k = 0;
    for (; k < nk; ++k) {
        if (!pipe.wait(k)) {
            dead = true;
            break;
        }
        const int phys = __shfl_sync(0xffffffffu, pipe.my_phys, k);
        if (phys >= 0) {
            const int base = w.block(v_begin + warp + k * NW) * kBlock;
            // tokens of the block that no row sees: from nvalid on, and h0 .. h1 - 1
            const int nvalid = min(kBlock, w.L - base);
            const int h0 = max(wa.num_sinks - base, 0), h1 = min(w.lo - base, kBlock);
            uint8_t *kt = pipe.ring + (k % STAGES) * Pipe::kStage;
            uint8_t *vt = kt + Pipe::kTile;
            const uint32_t kt_s = smem_addr(kt), vt_s = smem_addr(vt);
            float sf[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sf[nt][0] = sf[nt][1] = sf[nt][2] = sf[nt][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                uint32_t af[4];
                ldmatrix_x4(af, kt_s + tile_off(ka_row, 2 * kk + ka_half));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) Mma<T>::run(sf[nt], af, qf[nt][kk][0], qf[nt][kk][1]);
            }
            // sf[nt]: (token g, row 2c), (g, 2c+1), (g+8, 2c), (g+8, 2c+1)
            const bool v0 = g < nvalid && !(g >= h0 && g < h1);
            const bool v1 = g + 8 < nvalid && !(g + 8 >= h0 && g + 8 < h1);
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    bool s0 = v0, s1 = v1;
                    if constexpr (CHUNK) {
                        const int k0 = base + g, k1 = base + g + 8, pp = pos[nt][j];
                        s0 = k0 <= pp && (pp - k0 < wa.window || k0 < wa.num_sinks);
                        s1 = k1 <= pp && (pp - k1 < wa.window || k1 < wa.num_sinks);
                    }
                    const float x0 = s0 ? sf[nt][j] * a.scale_log2 : -INFINITY;
                    const float x1 = s1 ? sf[nt][j + 2] * a.scale_log2 : -INFINITY;
                    float bm = fmaxf(x0, x1);
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
                    const float m_new = fmaxf(mrow[nt][j], bm);
                    // a chunk's row may see nothing of the blocks so far
                    const float m_ref = CHUNK && m_new == -INFINITY ? 0.f : m_new;
                    const float alpha = fast_exp2(mrow[nt][j] - m_ref);
                    p[j] = fast_exp2(x0 - m_ref);
                    p[j + 2] = fast_exp2(x1 - m_ref);
                    lrow[nt][j] = lrow[nt][j] * alpha + p[j] + p[j + 2];
                    mrow[nt][j] = m_new;
#pragma unroll
                    for (int jj = 0; jj < KS; ++jj) {
                        acc[nt][jj][j] *= alpha;
                        acc[nt][jj][j + 2] *= alpha;
                    }
                }
                // P^T rounded to T for the tensor cores (the sum l keeps it in
                // f32): at most half a step of T relative per weight
                pb[nt][0] = movmatrix_trans(Mma<T>::pack(p[0], p[1]));
                pb[nt][1] = movmatrix_trans(Mma<T>::pack(p[2], p[3]));
            }
            if (nvalid < kBlock || h0 < h1) {
                // rows no query sees may hold anything (NaN included): zero them
                for (int idx = lane; idx < kBlock * (D / 8); idx += 32) {
                    const int t = idx / (D / 8), ch = idx % (D / 8);
                    if (t >= nvalid || (t >= h0 && t < h1))
                        *reinterpret_cast<uint4 *>(vt + tile_off(t, ch)) = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                uint32_t af[4];
                ldmatrix_x4_trans(af, vt_s + tile_off(va_row, 2 * j + va_half));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) Mma<T>::run(acc[nt][j], af, pb[nt][0], pb[nt][1]);
            }
        }
        __syncwarp();
        if (issued < nk) pipe.issue(issued++);
    }
    if (dead) pipe.drain(k, issued);

    // full row sums: add the partial sums of the 8 lanes that share c
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float v = lrow[nt][j];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            lrow[nt][j] = dead ? 0.f : v;
        }
    // the warp's ring is idle now: reuse it as [RMAX][D] fp32 scratch
    float *wacc = reinterpret_cast<float *>(pipe.ring);
    if (!dead) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = nt * 8 + 2 * c + (e & 1);
                    const int d = 16 * j + g + 8 * (e >> 1);
                    wacc[r * D + d] = acc[nt][j][e];
                }
    }
    if (g == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = nt * 8 + 2 * c + j;
                s_m[warp][r] = mrow[nt][j];
                s_l[warp][r] = lrow[nt][j];
            }
    }
    __syncthreads();

    const uint8_t *rings = align_smem_1024(dyn_smem);
    for (int idx = threadIdx.x; idx < rows * D; idx += NW * 32) {
        const int r = idx / D, d = idx % D;
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < NW; ++i)
            if (s_l[i][r] > 0.f) M = fmaxf(M, s_m[i][r]);
        float den = 0.f, o = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            if (s_l[i][r] > 0.f) {
                const float wt = fast_exp2(s_m[i][r] - M);
                den += wt * s_l[i][r];
                o += wt * reinterpret_cast<const float *>(rings + i * STAGES * Pipe::kStage)[r * D + d];
            }
        }
        o = den > 0.f ? o / den : 0.f;
        const size_t row = q_row(r);
        if (nparts == 1) {
            out[row * D + d] = narrow1(o, T());
        } else {
            a.ws_o[(row * a.num_parts + part) * D + d] = o;
            if (d == 0) a.ws_ml[row * a.num_parts + part] = make_float2(den > 0.f ? M : -INFINITY, den);
        }
    }
}

// Joins the partitions of one row with the four warps of a CTA: warp w takes
// every fourth partition and has eight of them in flight, and every warp works
// out all the weights.  merge_row's single warp takes partition after
// partition, about 10 us for the 65 of one 8192-token window.
template <typename T, int D>
__device__ __forceinline__ void merge_row_cta(const DecodeArgs &a, size_t row, int nparts) {
    constexpr int D4 = D / 4, PER = 32 / kMergeRows;
    __shared__ float4 s_acc[kMergeRows][D4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float2 *ml = a.ws_ml + row * a.num_parts;
    const float4 *op = reinterpret_cast<const float4 *>(a.ws_o + row * a.num_parts * D);
    float4 x[PER], acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto load = [&](int p0) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int p = p0 + warp + j * kMergeRows;
            if (p < nparts && lane < D4) x[j] = op[(size_t)p * D4 + lane];
        }
    };
    load(0);  // does not depend on the weights
    float M = -INFINITY, den = 0.f;
    for (int p = lane; p < nparts; p += 32) {
        const float2 v = ml[p];
        if (v.y > 0.f) M = fmaxf(M, v.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int p0 = 0; p0 < nparts; p0 += 32) {
        if (p0 > 0) load(p0);
        const float2 v = p0 + lane < nparts ? ml[p0 + lane] : make_float2(0.f, 0.f);
        const float w = v.y > 0.f ? v.y * fast_exp2(v.x - M) : 0.f;
        den += w;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, warp + j * kMergeRows);
            if (p0 + warp + j * kMergeRows < nparts && lane < D4) {
                acc.x += wj * x[j].x; acc.y += wj * x[j].y; acc.z += wj * x[j].z; acc.w += wj * x[j].w;
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (lane < D4) s_acc[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && lane < D4) {
#pragma unroll
        for (int w = 1; w < kMergeRows; ++w) {
            const float4 y = s_acc[w][lane];
            acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
        }
        const float inv = den > 0.f ? 1.f / den : 0.f;
        uint16_t *out = reinterpret_cast<uint16_t *>(a.out) + row * D + 4 * lane;
        const uint32_t lo = (uint32_t)narrow1(acc.x * inv, T()) | ((uint32_t)narrow1(acc.y * inv, T()) << 16);
        const uint32_t hi = (uint32_t)narrow1(acc.z * inv, T()) | ((uint32_t)narrow1(acc.w * inv, T()) << 16);
        *reinterpret_cast<uint2 *>(out) = make_uint2(lo, hi);
    }
}

// Joins the partitions of rows whose visible blocks were split: a row of q per
// warp, or per CTA when a row can have more than kMergeFew partitions.  Rows
// share their partitions with the other tokens of their tile (all of the
// sequence's, in decode_window_kernel).
template <typename T, int D, bool CHUNK>
__global__ void __launch_bounds__(kMergeRows * 32) merge_window_kernel(const WindowArgs wa) {
    const DecodeArgs &a = wa.d;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int lane = threadIdx.x & 31;
    const bool whole_cta = a.num_parts > kMergeFew;
    const size_t id = whole_cta ? blockIdx.x : (size_t)blockIdx.x * kMergeRows + (threadIdx.x >> 5);
    const size_t per_seq = (size_t)wa.max_query_len * a.num_q_heads;
    const int s = (int)(id / per_seq);
    if (s >= a.num_seqs) return;
    WindowSeq w;
    if (!window_seq<CHUNK>(wa, s, false, w)) return;
    const int i = (int)(id % per_seq) / a.num_q_heads;
    if (i >= w.n) return;
    if constexpr (CHUNK) {
        const int i0 = i / wa.tile_tokens * wa.tile_tokens;
        const int i1 = min(w.n - i0, wa.tile_tokens) + i0;
        window_blocks(w, w.L - w.n + i0, w.L - w.n + i1, wa.window, wa.num_sinks);
    }
    const int nparts = (w.nv + a.part_blocks - 1) / a.part_blocks;
    if (nparts <= 1) return;
    const size_t row = (size_t)(w.q0 + i) * a.num_q_heads + id % a.num_q_heads;
    if (whole_cta)
        merge_row_cta<T, D>(a, row, nparts);
    else
        merge_row<T, D>(a, row, nparts, lane);
}

}  // namespace pa
