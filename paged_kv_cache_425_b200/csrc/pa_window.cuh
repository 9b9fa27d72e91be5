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

#include <type_traits>

#include "pa_kernels.cuh"

namespace pa {

struct WindowArgs {
    DecodeArgs d;                // num_parts, part_blocks: of a run's visible blocks
    const int32_t *query_start;  // chunks only: [S + 1]
    int num_q_tokens;            // rows of q / out
    int max_query_len;           // 1 for decode
    int tile_tokens;             // query tokens that share one list of visible blocks
    int window;                  // >= 1
    int num_sinks;               // >= 0
    bool warp_runs;              // a warp per run
    int cluster;                 // CTAs per run, 0: d.num_parts partitions of d.part_blocks
};

// A run of query tokens of one sequence, and the blocks visible to it.
struct WindowSeq {
    int q0, n;       // first row of q / out (in tokens), query tokens
    int first, end;  // positions of the first query token and after the last
    int lo;          // first token inside any row's window
    int nsb;         // sink blocks in front of the window's blocks
    int skip;        // blocks between them, with no visible token
    int nv;          // visible blocks
    // logical block of visible block v
    __device__ __forceinline__ int block(int v) const { return v < nsb ? v : v + skip; }
};

__device__ __forceinline__ void window_blocks(WindowSeq &w, int first, int end, int window,
                                              int num_sinks) {
    w.first = first;
    w.end = end;
    w.lo = max(0, first - window + 1);
    const int b0 = w.lo / kBlock;
    w.nsb = min((min(num_sinks, end) + kBlock - 1) / kBlock, b0);
    w.skip = b0 - w.nsb;
    w.nv = (end + kBlock - 1) / kBlock - w.skip;
}

// The query tokens of sequence s's tile (decode: its one token); n = 0 if
// there are none.  Rows outside q / out and chunks longer than announced are
// reported and left out.
template <bool CHUNK>
__device__ __forceinline__ void window_seq(const WindowArgs &a, int s, int tile, bool report,
                                           WindowSeq &w) {
    if constexpr (!CHUNK) {
        const int L = clamp_context(a.d, s, report);
        w.q0 = s;
        w.n = L > 0 ? 1 : 0;
        window_blocks(w, L - w.n, L, a.window, a.num_sinks);
    } else {
        w.q0 = a.query_start[s];
        w.n = 0;
        int n = a.query_start[s + 1] - w.q0;
        int L = a.d.context_lens[s];
        const int cap = a.d.max_blocks_per_seq * kBlock;
        bool bad = L < 0 || L > cap || n < 0 || n > L;
        L = min(max(L, 0), cap);
        const bool outside = w.q0 < 0 || w.q0 > a.num_q_tokens || n > a.num_q_tokens - w.q0;
        n = min(max(n, 0), L);
        const bool drop = outside || n > a.max_query_len;
        if (report && (bad || drop)) flag_error(PA_DEVERR_CONTEXT_LEN);
        const int i0 = tile * a.tile_tokens;
        if (drop || i0 >= n) return;
        w.n = min(a.tile_tokens, n - i0);
        w.q0 += i0;
        window_blocks(w, L - n + i0, L - n + i0 + w.n, a.window, a.num_sinks);
    }
}

// ------------------------------------------------------------------ thread-block clusters
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
// With nothing to publish (the releasing form takes about 1000 cycles).
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Shared-memory address `addr` of this CTA, in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_store4(uint32_t addr, const float4 &v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w)
                 : "memory");
}

__device__ __forceinline__ void cluster_store2(uint32_t addr, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// ------------------------------------------------------------------ decode over the visible blocks
// WarpPipe that issues several blocks at once, each box (K and V, D / 64 each)
// from a lane of its own: one after the other by one lane, with a proxy fence
// per block, a block takes about 500 cycles to issue, which a warp with few
// others beside it waits for.  (With 24 warps per SM nobody waits for it, and
// the one lane is 3 % faster.)
template <int D, int STAGES>
struct WindowPipe : WarpPipe<D, STAGES> {
    using Base = WarpPipe<D, STAGES>;
    static constexpr int kBoxes = 2 * (D / 64);
    static_assert(STAGES * kBoxes <= 32, "a lane per box");
    // Blocks k .. k + n - 1 (n <= STAGES).  `reuse`: the stages were read
    // before, and those reads go first.
    __device__ __forceinline__ void issue(int k, int n, bool reuse) {
        const int sub = this->lane / kBoxes, box = this->lane % kBoxes;
        const int phys = __shfl_sync(0xffffffffu, this->my_phys, (k + sub) & 31);
        const bool mine = sub < n;
        uint64_t *b = &this->bar[(k + sub) % STAGES];
        if (mine && box == 0) {
            if (phys >= 0)
                mbar_arrive_expect_tx(b, Base::kStage);
            else
                mbar_arrive(b);  // bad id: the stage completes empty
        }
        __syncwarp();
        if (mine && phys >= 0) {
            const int col = box % (D / 64);
            const bool v = box >= D / 64;
            if (reuse) fence_proxy_async_smem();
            tma_load_2d_hint(this->ring + ((k + sub) % STAGES) * Base::kStage +
                                 (v ? Base::kTile : 0) + col * 2048,
                             v ? this->tmv : this->tmk, b, col * 64,
                             (phys * this->num_kv_heads + this->kvh) * kBlock, this->policy);
        }
    }
};

constexpr int kMaxCluster = 16;

__device__ __forceinline__ uint2 narrow4(const float4 &v, float inv, __half) {
    return make_uint2(Mma<__half>::pack(v.x * inv, v.y * inv), Mma<__half>::pack(v.z * inv, v.w * inv));
}
__device__ __forceinline__ uint2 narrow4(const float4 &v, float inv, __nv_bfloat16) {
    return make_uint2(Mma<__nv_bfloat16>::pack(v.x * inv, v.y * inv),
                      Mma<__nv_bfloat16>::pack(v.z * inv, v.w * inv));
}

// Grid: x = sequence * Hkv + kv head, y = partition of its visible blocks,
// z = run of tile_tokens query tokens (chunks); WARP: x = NW runs.  NT 8-row column tiles: rows of
// a run (tokens x group) <= 8 * NT.
//
// A warp takes every NW-th block of its CTA's blocks, U per step, and has
// STAGES in flight.  Five shapes:
//  * many rows (U = 1): 4 warps with one block each (two at head_dim 64), six
//    CTAs per SM, partitions of PB blocks: the shape that reaches the memory's
//    bandwidth best once the GPU is full.
//  * fewer (U = 2, PB = 0: a CTA takes its whole run): 4 warps with three
//    blocks, two CTAs per SM, for runs that fit in one such wave.  At one block
//    per step a warp needs about 1300 cycles for the chain from scores to
//    weights, which only many warps hide; two blocks are two chains.
//  * at most a run per SM (U = 2, PB = 0, no cluster): the same with 6 or 8 warps,
//    one CTA per SM (144 runs of 33 blocks 7.5 us, 10.3 with four warps; of 180
//    blocks 36.0, 39.5 in partitions).
//  * few rows (CLUSTER): the gridDim.y CTAs of a run, 6 or 8 warps each, form one
//    thread-block cluster, take an equal share of its blocks each and send
//    their results to each other's shared memory: one launch, no workspace.
// Measured (bf16, 32 heads on 8, head_dim 128): 128 sequences with 4096-token
// windows 311 us, 2.16 GB of visible rows at 6.9 TB/s (a copy reaches 6.55; L2
// keeps a part between calls); 32 with 512-token windows, one wave, 10.9 us (15.8
// in partitions); one with an 8192-token window in clusters of ten 10.4 us (13.5
// in partitions).
//  * many short runs (WARP, U = 1): a warp takes a whole run, four runs per CTA,
//    with nothing to join: a CTA per run spends most of its 3 us waiting when the
//    run is a few blocks (7360 runs of one block: 40 us, 18 here).
// Partitions are joined by merge_window_kernel through the workspace.
template <typename T, int D, int NW, int STAGES, int U, int PB, int NT, bool CHUNK, bool CLUSTER, bool WARP>
__global__ void __launch_bounds__(NW * 32, U > 1 ? 1 : NT == 1 ? PA_DECODE_MIN_CTAS : 3)
    decode_window_kernel(const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv, const WindowArgs wa) {
    using Pipe = std::conditional_t<U == 1, WarpPipe<D, STAGES>, WindowPipe<D, STAGES>>;
    const DecodeArgs &a = wa.d;
    constexpr int KS = D / 16;          // 16-wide steps of the head dim
    constexpr int RMAX = 8 * NT;        // rows this build handles
    constexpr int D4 = D / 4;
    static_assert(RMAX * D * 4 <= STAGES * Pipe::kStage, "combine scratch fits in a warp ring");
    static_assert(kMaxCluster <= D4, "one thread per row and peer sends the row's max and sum");
    extern __shared__ uint8_t dyn_smem[];
    __shared__ __align__(8) uint64_t bars[NW][STAGES];
    __shared__ float s_m[NW][RMAX], s_l[NW][RMAX];
    // what the cluster's CTAs send here: this CTA's share of the rows' elements
    // from each of them, and every row's (max, sum)
    __shared__ __align__(16) float4 r_o[CLUSTER ? RMAX * D4 + kMaxCluster : 1];
    __shared__ __align__(8) float2 r_ml[CLUSTER ? kMaxCluster * RMAX : 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.y;
    int kvh = blockIdx.x % a.num_kv_heads, s = blockIdx.x / a.num_kv_heads, tile = blockIdx.z;
    if constexpr (WARP) {  // runs in the order kv head, run of the sequence, sequence
        const long long id = (long long)blockIdx.x * NW + warp;
        const int tiles = CHUNK ? (wa.max_query_len + wa.tile_tokens - 1) / wa.tile_tokens : 1;
        kvh = (int)(id % a.num_kv_heads);
        tile = (int)(id / a.num_kv_heads % tiles);
        const long long seq = id / a.num_kv_heads / tiles;
        if (seq >= a.num_seqs) return;
        s = (int)seq;
    }
    const int G = a.num_q_heads / a.num_kv_heads;
    pdl_launch_dependents();
    pdl_wait_prior();
    WindowSeq w;
    window_seq<CHUNK>(wa, s, tile, part == 0 && kvh == 0 && tile == 0 && (WARP ? lane : threadIdx.x) == 0, w);
    uint16_t *out = reinterpret_cast<uint16_t *>(a.out);
    // row r of the run -> row of q / out
    auto q_row = [&](int r) {
        return CHUNK ? (size_t)(w.q0 + r / G) * a.num_q_heads + (size_t)kvh * G + r % G
                     : (size_t)s * a.num_q_heads + (size_t)kvh * G + r;
    };
    if (w.n == 0) {  // the same for every CTA of a cluster
        if (!CHUNK && part == 0)
            for (int i = WARP ? lane : threadIdx.x; i < G * D; i += WARP ? 32 : NW * 32)
                out[q_row(0) * D + i] = 0;
        return;
    }
    if constexpr (CLUSTER) cluster_arrive_relaxed();  // waited for before the first remote store
    const int rows = CHUNK ? w.n * G : G;
    const int share = CLUSTER ? (w.nv + (int)gridDim.y - 1) / (int)gridDim.y
                              : PB > 0 ? PB : w.nv;  // blocks per CTA
    const int nparts = (w.nv + share - 1) / share;
    if (!CLUSTER && part >= nparts) return;
    const int v_begin = part * share;
    const int nv_local = max(min(share, w.nv - v_begin), 0);
    constexpr int STEP = WARP ? 1 : NW;  // the warp's k-th block is w0 + k * STEP
    const int w0 = WARP ? 0 : warp;
    const int nk = warp_block_count(nv_local, w0, STEP);

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
            a.block_tables[(size_t)s * a.max_blocks_per_seq + w.block(v_begin + w0 + lane * STEP)];
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
    if (!CHUNK && a.k_new != nullptr && a.context_lens[s] == w.end) {
        const int li = w.nv - 1 - v_begin;
        if (li >= 0 && li < nv_local && li % STEP == w0) k_app = li / STEP;
    }
    if (k_app >= 0 && k_app < issued) append_new_token<D>(a, s, kvh, w.end, lane);
    if constexpr (U > 1)
        pipe.issue(0, issued, false);
    else
        for (int k = 0; k < issued; ++k) pipe.issue(k);
    if (k_app >= issued) append_new_token<D>(a, s, kvh, w.end, lane);

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
            for (int j = 0; j < 2; ++j) pos[nt][j] = w.first + min(nt * 8 + 2 * c + j, rows - 1) / G;
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
    for (; k < nk; k += U) {
        bool ok = true;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k + u < nk) ok = pipe.wait(k + u) && ok;
        if (!ok) {
            dead = true;
            break;
        }
        bool use[U], any = false;
        int base[U], nvalid[U], h0[U], h1[U];
        uint8_t *kt[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            use[u] = k + u < nk && __shfl_sync(0xffffffffu, pipe.my_phys, k + u) >= 0;
            any = any || use[u];
            base[u] = w.block(v_begin + w0 + (k + u) * STEP) * kBlock;
            // tokens of the block that no row sees: from nvalid on, and h0 .. h1 - 1
            nvalid[u] = min(kBlock, w.end - base[u]);
            h0[u] = max(wa.num_sinks - base[u], 0);
            h1[u] = min(w.lo - base[u], kBlock);
            kt[u] = pipe.ring + ((k + u) % STAGES) * Pipe::kStage;
        }
        if (any) {
            float sf[U][NT][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    sf[u][nt][0] = sf[u][nt][1] = sf[u][nt][2] = sf[u][nt][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    // (an unused block's stage holds anything: its scores are masked)
                    uint32_t af[4];
                    ldmatrix_x4(af, smem_addr(kt[u]) + tile_off(ka_row, 2 * kk + ka_half));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        Mma<T>::run(sf[u][nt], af, qf[nt][kk][0], qf[nt][kk][1]);
                }
            // sf[u][nt]: (token g, row 2c), (g, 2c+1), (g+8, 2c), (g+8, 2c+1)
            bool v0[U], v1[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v0[u] = use[u] && g < nvalid[u] && !(g >= h0[u] && g < h1[u]);
                v1[u] = use[u] && g + 8 < nvalid[u] && !(g + 8 >= h0[u] && g + 8 < h1[u]);
            }
            uint32_t pb[U][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[U][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float bm = -INFINITY;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        bool s0 = v0[u], s1 = v1[u];
                        if constexpr (CHUNK) {
                            const int k0 = base[u] + g, k1 = base[u] + g + 8, pp = pos[nt][j];
                            s0 = use[u] && k0 <= pp && (pp - k0 < wa.window || k0 < wa.num_sinks);
                            s1 = use[u] && k1 <= pp && (pp - k1 < wa.window || k1 < wa.num_sinks);
                        }
                        p[u][j] = s0 ? sf[u][nt][j] * a.scale_log2 : -INFINITY;
                        p[u][j + 2] = s1 ? sf[u][nt][j + 2] * a.scale_log2 : -INFINITY;
                        bm = fmaxf(bm, fmaxf(p[u][j], p[u][j + 2]));
                    }
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
                    const float m_new = fmaxf(mrow[nt][j], bm);
                    // no score above -infinity so far (a visible key may give it,
                    // and a chunk's row may see nothing of the blocks so far)
                    const float m_ref = m_new == -INFINITY ? 0.f : m_new;
                    const float alpha = fast_exp2(mrow[nt][j] - m_ref);
                    float sum = 0.f;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        p[u][j] = fast_exp2(p[u][j] - m_ref);
                        p[u][j + 2] = fast_exp2(p[u][j + 2] - m_ref);
                        sum += p[u][j] + p[u][j + 2];
                    }
                    lrow[nt][j] = lrow[nt][j] * alpha + sum;
                    mrow[nt][j] = m_new;
#pragma unroll
                    for (int jj = 0; jj < KS; ++jj) {
                        acc[nt][jj][j] *= alpha;
                        acc[nt][jj][j + 2] *= alpha;
                    }
                }
                // P^T rounded to T for the tensor cores (the sum l keeps it in
                // f32): at most half a step of T relative per weight
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    pb[u][nt][0] = movmatrix_trans(Mma<T>::pack(p[u][0], p[u][1]));
                    pb[u][nt][1] = movmatrix_trans(Mma<T>::pack(p[u][2], p[u][3]));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!use[u]) continue;
                uint8_t *vt = kt[u] + Pipe::kTile;
                if (nvalid[u] < kBlock || h0[u] < h1[u]) {
                    // rows no query sees may hold anything (NaN included): zero them
                    for (int idx = lane; idx < kBlock * (D / 8); idx += 32) {
                        const int t = idx / (D / 8), ch = idx % (D / 8);
                        if (t >= nvalid[u] || (t >= h0[u] && t < h1[u]))
                            *reinterpret_cast<uint4 *>(vt + tile_off(t, ch)) = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
                const uint32_t vt_s = smem_addr(vt);
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    uint32_t af[4];
                    ldmatrix_x4_trans(af, vt_s + tile_off(va_row, 2 * j + va_half));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        Mma<T>::run(acc[nt][j], af, pb[u][nt][0], pb[u][nt][1]);
                }
            }
        }
        __syncwarp();
        if constexpr (U > 1) {
            const int n = min(U, nk - issued);
            if (n > 0) pipe.issue(issued, n, true);
            issued += n;
        } else if (issued < nk) {
            pipe.issue(issued++);
        }
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
    if constexpr (WARP) {  // the warp has its rows complete
        __syncwarp();
        for (int e = lane; e < rows * D4; e += 32) {
            const int r = e / D4, d4 = e % D4;
            const float den = s_l[warp][r];
            const float4 o = has_weight(den) ? reinterpret_cast<const float4 *>(wacc)[e]
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<uint2 *>(out + q_row(r) * D + d4 * 4) =
                narrow4(o, has_weight(den) ? 1.f / den : 0.f, T());
        }
        return;
    }
    __syncthreads();

    const uint8_t *rings = align_smem_1024(dyn_smem);
    const int total = rows * D4;               // float4 pieces of the rows
    const int ctas = gridDim.y;
    const int slots = CLUSTER ? (total + ctas - 1) / ctas : 1;  // pieces each CTA joins
    if constexpr (CLUSTER) cluster_wait();     // every CTA of the cluster runs by now
    for (int e = threadIdx.x; e < total; e += NW * 32) {
        const int r = e / D4, d4 = e % D4;
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < NW; ++i)
            if (has_weight(s_l[i][r])) M = fmaxf(M, s_m[i][r]);
        float den = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            if (has_weight(s_l[i][r])) {
                const float wt = fast_exp2(s_m[i][r] - M);
                const float4 x = reinterpret_cast<const float4 *>(rings + i * STAGES * Pipe::kStage)[e];
                den += wt * s_l[i][r];
                o.x += wt * x.x; o.y += wt * x.y; o.z += wt * x.z; o.w += wt * x.w;
            }
        }
        const float inv = has_weight(den) ? 1.f / den : 0.f;
        if constexpr (CLUSTER) {
            // unnormalised, with the CTA's max and sum, to the CTA that joins it
            cluster_store4(cluster_addr(smem_addr(&r_o[part * slots + e % slots]), e / slots), o);
            if (d4 < ctas) cluster_store2(cluster_addr(smem_addr(&r_ml[part * RMAX + r]), d4), M, den);
        } else {
            const size_t row = q_row(r);
            if (nparts == 1) {
                *reinterpret_cast<uint2 *>(out + row * D + d4 * 4) = narrow4(o, inv, T());
            } else {
                o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
                reinterpret_cast<float4 *>(a.ws_o)[(row * a.num_parts + part) * D4 + d4] = o;
                if (d4 == 0)
                    a.ws_ml[row * a.num_parts + part] = make_float2(has_weight(den) ? M : -INFINITY, den);
            }
        }
    }
    if constexpr (CLUSTER) {
        cluster_arrive();
        cluster_wait();
        for (int i = threadIdx.x; i < slots; i += NW * 32) {
            const int e = part * slots + i;
            if (e >= total) break;
            const int r = e / D4, d4 = e % D4;
            float M = -INFINITY, den = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int p = 0; p < ctas; ++p) M = fmaxf(M, r_ml[p * RMAX + r].x);
            for (int p = 0; p < ctas; ++p) {
                const float2 ml = r_ml[p * RMAX + r];
                const float4 x = r_o[p * slots + i];
                const float wt = has_weight(ml.y) ? fast_exp2(ml.x - M) : 0.f;
                den += wt * ml.y;
                o.x += wt * x.x; o.y += wt * x.y; o.z += wt * x.z; o.w += wt * x.w;
            }
            *reinterpret_cast<uint2 *>(out + q_row(r) * D + d4 * 4) =
                narrow4(o, has_weight(den) ? 1.f / den : 0.f, T());
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
        if (has_weight(v.y)) M = fmaxf(M, v.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int p0 = 0; p0 < nparts; p0 += 32) {
        if (p0 > 0) load(p0);
        const float2 v = p0 + lane < nparts ? ml[p0 + lane] : make_float2(0.f, 0.f);
        const float w = has_weight(v.y) ? v.y * fast_exp2(v.x - M) : 0.f;
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
        const float inv = has_weight(den) ? 1.f / den : 0.f;
        uint16_t *out = reinterpret_cast<uint16_t *>(a.out) + row * D + 4 * lane;
        const uint32_t lo = (uint32_t)narrow1(acc.x * inv, T()) | ((uint32_t)narrow1(acc.y * inv, T()) << 16);
        const uint32_t hi = (uint32_t)narrow1(acc.z * inv, T()) | ((uint32_t)narrow1(acc.w * inv, T()) << 16);
        *reinterpret_cast<uint2 *>(out) = make_uint2(lo, hi);
    }
}

// Joins the partitions of rows whose visible blocks were split: a row of q per
// warp, or per CTA when a row can have more than kMergeFew partitions.  Rows
// share their partitions with the other tokens of their run of tile_tokens.
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
    int i = (int)(id % per_seq) / a.num_q_heads;
    const int tile = CHUNK ? i / wa.tile_tokens : 0;
    i -= tile * wa.tile_tokens;
    window_seq<CHUNK>(wa, s, tile, false, w);
    if (i >= w.n) return;
    const int nparts = (w.nv + a.part_blocks - 1) / a.part_blocks;
    if (nparts <= 1) return;
    const size_t row = (size_t)(w.q0 + i) * a.num_q_heads + id % a.num_q_heads;
    if (whole_cta)
        merge_row_cta<T, D>(a, row, nparts);
    else
        merge_row<T, D>(a, row, nparts, lane);
}

}  // namespace pa
