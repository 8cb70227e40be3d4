// kv4_attn.cuh -- softmax attention of a ragged batch of queries over the
// paged 4-bit cache (kv4_cache.cuh), for few query rows per request: decode
// steps and short drafts.
//     o_i = sum_j softmax_j(scale q_i . k_j) v_j  over the keys j that query i
//     may see (j <= pos_i when causal, j > pos_i - window when windowed)
//
// Rows.  The group = q_heads / kv_heads query heads that share a key/value head
// are packed with the request's query tokens into rows (token * group + head),
// so a cached token is read and decoded once for all rows of a tile (4, 8, 16
// or 24).
//
// Bound: HBM.  A cached token of a head costs 2 * (D/2 + D/16) bytes (144 at
// D = 128) and 4 * D * rows flop, far below the tensor cores' balance, so the
// contractions run on mma.sync (m16n8k16) only to keep the issue slots for the
// decoding: per pair of codes a shift (for three of four), a logic op, a packed
// subtraction and a packed product (kv4_pair).  The rows are the MMA's narrow side, and the operand orders are
// chosen so that the packed words need no reordering:
//   S^T = K Q^T: A = 16 tokens.  Thread (g, t) holds tokens g and g + 8 and their
//     channels [32t, 32t + 32) (D = 128): 16 bytes of codes and one step each;
//     word w's pairs (0,4)(1,5) and (2,6)(3,7) are two MMAs, and q is loaded
//     once in that order.
//   O^T = V^T P^T: A = 16 channels x 16 tokens.  Thread (g, t) holds channels
//     [16g, 16g + 16) of the tokens (2t, 2t+1), (2t+8, 2t+9); a byte permute
//     pairs two tokens' words and the same decode gives the (token, token + 1)
//     pairs of each channel.  P comes from S's accumulators by movmatrix, and
//     a thread's outputs are 16 consecutive channels of two rows.
// P is rounded to bf16 (at most 2^-8 of each weight; the row sum adds the
// unrounded weights); a tile of 4 rows uses the other 4 columns of the MMA for
// what that rounding left, so its weights enter with 16 bits.  Scores,
// statistics and outputs are float32.
//
// Work split.  A unit is (request, kv head, row tile, chunk of 128 tokens); the
// units of the whole ragged batch form one list (from the lengths, on the
// device) that is cut into equal ranges, one per CTA, so a long request spreads
// over the GPU and a batch of ragged ones leaves no CTA idle.  A tile cut
// between CTAs leaves (max, sum, unnormalised output) of each piece in the
// workspace, and kv4_combine_kernel joins them in order (no atomics: the result
// does not depend on timing).
//
// Data movement.  A producer warp streams each unit's pages into a ring, the
// codes with untiled bulk copies (one per page: a page's head is contiguous),
// the steps with 16-byte copies of its lanes, and writes which of the 128 tokens
// exist: tokens past the length, of pages
// that the table does not name, or that no query of the request can see any
// more are never attended to, and their steps are taken as 0, whatever bytes
// lie there.  Four consumer warps take 32 tokens each with statistics of their
// own, joined at the end of a tile's piece.
//
// Measured on a B200 (calls replayed from a graph, 32/8 heads of 128): 64 requests
// of 511 to 8200 tokens, 98 us = 3.3 TB/s (323 MB, 50 us at the copy rate), one of
// 131,071 tokens 51.5 us (23), one of 999 in clusters 7.0 us.  What bounds the first is
// latency: 223 warp instructions per 8 tokens and head would take 57 us issued without
// gaps, but 12 consumer warps a SM, each with one dependent chain from the codes to the
// second product, fill 66% of the issue slots (ALU pipe 58%, FMA 45%, HBM 51%).  An
// earlier form with 200 instructions took 95 us, 89 without the copies and 58 without
// the arithmetic.  Tried on that form and slower: rows on the MMA's wide side (136 us),
// two CTAs per SM (101), shifts by multiplication (97); four CTAs per SM: the same.
#pragma once

#include <cuda_bf16.h>

#include "device_common.cuh"
#include "kv4_cache.cuh"
#include "w4a16_gemv.cuh"

namespace qat4 {

constexpr int kKaWarps = 4;                       // consumer warps
constexpr int kKaThreads = 32 * (kKaWarps + 1);   // + one producer warp
constexpr int kKaChunk = 128;                     // tokens per unit
constexpr float kKaGrow = 8.0f;   // a row's reference maximum moves only when exceeded by 2^8
// Units after which a tile's rows so far are joined into the CTA's piece in the workspace, and its sums start anew.
// The tensor cores cut what they add to the bits of the running sum: over n tokens of a warp of like weights the
// output comes out low by n 2^-27.5 of itself (measured: 4.6e-3 after 2^20 tokens a warp), by 2^-12.5 after the 2^15
// here (measured: 1.5e-4).
constexpr int kKaFold = 1024;
static_assert((kKaFold & (kKaFold - 1)) == 0, "a power of two");

struct AttnParams {
    const uint16_t* q;        // [N, Hq, D], token stride q_stride
    int64_t q_stride;
    const int* table;
    int64_t table_stride;
    const int* seq_lens;
    const int* cu_q;
    uint16_t* out;            // [N, Hq, D]
    float* lse;               // [N, Hq] or null
    float* part;              // workspace: pieces of cut tiles
    int4* meta;               // workspace: two records per CTA
    Kv4View c;
    int N, B, Hq, group, max_blocks, causal, window;
    int rows_lo, rows_hi;     // this kernel takes requests with rows_lo <= query rows per kv head <= rows_hi
    float scale_log2;         // scale * log2(e)
    uint64_t limit_ns;
};

// One request as the kernels see it (lengths cut to what the table and q can hold).
struct Request {
    int q0, nq;       // first query row of q and number of query tokens
    int len;          // cached tokens
    int first;        // position of the first query token (may be negative: then it sees nothing)
    int lo;           // first token any query can see
};
__device__ __forceinline__ Request kv4_request(const AttnParams& p, int b) {
    Request r;
    const int a = min(max(kv4_ld(p.cu_q + b), 0), p.N), e = min(max(kv4_ld(p.cu_q + b + 1), 0), p.N);
    r.q0 = a;
    r.nq = max(0, e - a);
    const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.c.page;
    const int len = max(0, kv4_ld(p.seq_lens + b));
    r.len = static_cast<int>(len < cap ? len : cap);
    r.first = r.len - r.nq;
    r.lo = p.window > 0 ? max(0, r.first - p.window + 1) : 0;
    return r;
}

template <int ROWS>
struct Units {
    int tiles, chunks, c0;    // row tiles, chunks per tile, first chunk
};
template <int ROWS>
__device__ __forceinline__ Units<ROWS> kv4_units(const AttnParams& p, const Request& r) {
    Units<ROWS> u;
    const int64_t rows = static_cast<int64_t>(r.nq) * p.group;
    const bool mine = rows >= p.rows_lo && rows <= p.rows_hi;
    u.tiles = mine ? static_cast<int>((rows + ROWS - 1) / ROWS) : 0;
    u.c0 = r.lo / kKaChunk;
    const int n = (r.len + kKaChunk - 1) / kKaChunk - u.c0;
    u.chunks = n > 1 ? n : 1;            // an empty request still writes its rows
    return u;
}

// A place in the unit list: request b, kv head, row tile and chunk.
template <int ROWS>
struct Place {
    Request r;
    Units<ROWS> un;
    int b, kvh, tile, ch;
    __device__ __forceinline__ void start(const AttnParams& p, int b_, int64_t skip) {
        b = b_;
        r = kv4_request(p, b);
        un = kv4_units<ROWS>(p, r);
        // 64-bit divisions only where a request has that many units
        if (skip <= 0x7fffffff) {
            const uint32_t s = static_cast<uint32_t>(skip), t = s / static_cast<uint32_t>(un.chunks);
            ch = static_cast<int>(s - t * un.chunks);
            kvh = static_cast<int>(t / static_cast<uint32_t>(un.tiles));
            tile = static_cast<int>(t - kvh * un.tiles);
        } else {
            const int64_t t = skip / un.chunks;
            ch = static_cast<int>(skip - t * un.chunks);
            kvh = static_cast<int>(t / un.tiles);
            tile = static_cast<int>(t - static_cast<int64_t>(kvh) * un.tiles);
        }
    }
    // the next unit; `more`: there is one
    __device__ __forceinline__ void next(const AttnParams& p, bool more) {
        if (++ch < un.chunks) return;
        ch = 0;
        if (++tile < un.tiles) return;
        tile = 0;
        if (++kvh < p.c.heads || !more) return;
        kvh = 0;
        do {
            ++b;
            r = kv4_request(p, b);
            un = kv4_units<ROWS>(p, r);
        } while (un.tiles == 0);
    }
    __device__ __forceinline__ int t0() const { return (un.c0 + ch) * kKaChunk; }
};

template <int D, int ROWS>
struct KaLayout {
    static constexpr int kCodes = kKaChunk * D / 2;
    static constexpr int kSteps = kKaChunk * (D / 32) * 2;
    static constexpr int kStage = 2 * kCodes + 2 * kSteps;
    static constexpr int kN = (ROWS + 7) / 8;                     // MMA column tiles of 8 rows
    static constexpr bool kQShared = ROWS == 24;                  // q in shared memory, where registers run out
    static constexpr int kPass = kQShared && D == 128 ? 1 : 2;    // tiles of 16 tokens of a warp at once
    static constexpr int kPerSm = ROWS >= 16 ? 2 : 3;             // CTAs per SM (registers, shared memory)
    static constexpr int kStages = ROWS == 16 ? 4 : 3;            // 73 or 55 KB of ring at D = 128
    static constexpr int kORow = D * 4 + 16;                      // bytes of an output row in the join buffer
    static constexpr int kJoin = kKaWarps * ROWS * kORow;
    static constexpr int kQ = kQShared ? kN * (D / 16) * 32 * 8 : 0;
    static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStage + kJoin + kQ;
};

// Workspace floats of one piece: ROWS rows of D outputs, then ROWS maxima (log2) and ROWS sums.
template <int D, int ROWS>
__host__ __device__ constexpr int ka_piece() { return ROWS * (D + 2); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// log-sum-exp of a row from its reference maximum (log2) and sum: -infinity where no key was seen, NaN where a
// score was.
__device__ __forceinline__ float kv4_lse(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Row `row` of a tile's result: out (and lse) from the unnormalised sums.
__device__ __forceinline__ int64_t ka_out_row(const AttnParams& p, const Request& r, int kvh, int row) {
    const int tok = row / p.group;
    return static_cast<int64_t>(r.q0 + tok) * p.Hq + kvh * p.group + (row - tok * p.group);
}

// gm_mma with a zero accumulator.
__device__ __forceinline__ void ka_mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Transposes an 8 x 8 matrix of 16-bit values held as one row pair per lane.
__device__ __forceinline__ uint32_t ka_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}

// CL: a cluster of kKaCluster CTAs per row tile, its chunks cut evenly and the pieces joined through
// the cluster's shared memory: one launch and no workspace, for batches too small to fill the GPU.
// Otherwise the stream of all units is cut evenly over the grid.
constexpr int kKaCluster = 8;
// Tiles that come in clusters: batches with tiles of 24 rows fill the GPU.
__host__ __device__ constexpr bool ka_clusters(int rows) { return rows < 24; }

// FOLD: a CTA may have more than kKaFold units of one tile; where the call's sizes rule that out, the kernel is built
// without the fold, whose registers cost tiles of 16 rows 3% (64 requests of 16 rows 154 us, 159 with it).
template <int D, int ROWS, bool CL, bool FOLD>
__global__ void __launch_bounds__(kKaThreads, KaLayout<D, ROWS>::kPerSm)
kv4_decode_kernel(const AttnParams p) {
    static_assert(!CL || (ka_clusters(ROWS) && !FOLD), "no call has such clusters");
    using L = KaLayout<D, ROWS>;
    constexpr int kStages = L::kStages;
    constexpr bool kLo = ROWS == 4;            // columns 4..7 carry the weights' rounding remainders
    constexpr int kN = L::kN;
    constexpr bool kQs = L::kQShared;
    constexpr int kPass = L::kPass;
    constexpr int kW = D / 32;                 // words of a thread's key channels (4 or 2)
    constexpr int kVW = D / 64;                // words of a thread's value channels (2 or 1)
    constexpr int kM = D / 16;                 // output tiles of 16 channels
    extern __shared__ __align__(128) uint8_t ka_smem[];
    __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages];
    __shared__ uint32_t live_bits[kStages][4];
    __shared__ float join_m[kKaWarps][24], join_l[kKaWarps][24];
    __shared__ __align__(16) float res[CL ? ka_piece<D, ROWS>() : 4];
    __shared__ int64_t scan[32], s_skip;
    __shared__ int s_b;
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();

    // ---- this CTA's range of the unit list (of the tile list, in clusters)
    auto count = [&](int b) -> int64_t {
        const Units<ROWS> u = kv4_units<ROWS>(p, kv4_request(p, b));
        return static_cast<int64_t>(u.tiles) * (CL ? 1 : u.chunks) * p.c.heads;
    };
    const int per = (p.B + kKaThreads - 1) / kKaThreads;
    const int rb0 = min(p.B, tid * per), rb1 = min(p.B, rb0 + per);
    int64_t mine = 0;
    for (int b = rb0; b < rb1; ++b) mine += count(b);
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += a;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) {
        s_b = -1;
        abort_flag = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full_bar[s], 33);            // the producer's codes, and each of its lanes' steps
            mbar_init(&empty_bar[s], kKaWarps);
        }
        fence_mbar_init();
    }
    if (!CL && tid < 2) p.meta[2 * blockIdx.x + tid] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int w = 0; w <= kKaWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    int64_t u0, u1;
    if (CL) {
        u0 = blockIdx.x / kKaCluster;
        u1 = u0 < total ? u0 + 1 : u0;
    } else {
        const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);     // every CTA of these has work
        // range i starts at floor(total i / ctas), without 64-bit divisions while there are few units
        const uint32_t n = max(1u, static_cast<uint32_t>(ctas)), i = blockIdx.x;
        const int64_t each = total <= 0x7fffffff ? static_cast<uint32_t>(total) / n : total / n;
        const uint32_t more = static_cast<uint32_t>(total - each * n);
        u0 = i < ctas ? each * i + more * i / n : 0;
        u1 = i < ctas ? each * (i + 1) + more * (i + 1) / n : 0;
    }
    if (u0 < u1 && u0 >= before && u0 < before + mine) {
        int64_t at = before;
        for (int b = rb0; b < rb1; ++b) {
            const int64_t n = count(b);
            if (u0 < at + n) {
                s_b = b;
                s_skip = u0 - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    if (u0 >= u1) return;                       // in clusters: every CTA of it
    volatile int* abort = &abort_flag;
    const uint32_t ring = smem_u32(ka_smem);
    Place<ROWS> at;
    if (CL) {
        const int rank = static_cast<int>(cluster_ctarank());
        at.b = s_b;
        at.r = kv4_request(p, at.b);
        at.un = kv4_units<ROWS>(p, at.r);
        at.kvh = static_cast<int>(s_skip / at.un.tiles);
        at.tile = static_cast<int>(s_skip % at.un.tiles);
        at.ch = at.un.chunks * rank / kKaCluster;
        u0 = 0;
        u1 = at.un.chunks * (rank + 1) / kKaCluster - at.ch;      // none for some ranks of a short request
    } else {
        at.start(p, s_b, s_skip);
    }
    const int page = p.c.page, sh = __ffs(page) - 1;

    if (warp == kKaWarps) {
        // ------------------------------------------------------------ producer
        const int np = kKaChunk >> sh;                         // pages per chunk, 1..8
        const bool vals = lane >= np, has = lane < 2 * np;     // lane's page of the key codes, then of the value codes
        const int pi = vals ? lane - np : lane;
        const uint32_t dst0 = (vals ? L::kCodes : 0) + pi * page * (D / 2);
        // this lane's entry of the block table for a unit, -1 where nothing is to be copied; loaded one unit
        // ahead, so that its latency is not part of the ring's round trip
        auto entry = [&](const Place<ROWS>& x) -> int {
            const int pt = x.t0() + pi * page;                 // first token of this lane's page
            // pt < len keeps the index inside the table's row
            return has && pt < x.r.len && pt + page > x.r.lo ? kv4_ld(p.table + x.b * p.table_stride + (pt >> sh)) : -1;
        };
        int64_t issued = 0;
        int s = 0;
        uint32_t ph = 0;
        int id = u0 < u1 ? entry(at) : -1;
        for (int64_t u = u0; u < u1; ++u) {
            Place<ROWS> ahead = at;
            ahead.next(p, u + 1 < u1);
            const int id_next = u + 1 < u1 ? entry(ahead) : -1;
            int ok = 1;
            if (lane == 0) ok = kv4_wait(&empty_bar[s], ph ^ 1u, abort, p.limit_ns) ? 1 : 0;
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            if (id >= p.c.pages) id = -1;
            const int t0 = at.t0(), pt = t0 + pi * page;
            // tokens that exist, 32 per word in lanes 0..3: inside [lo, len) and of a page that exists
            const uint32_t ids = __ballot_sync(0xffffffffu, !vals && id >= 0);
            if (lane < 4) {
                const int w0 = t0 + 32 * lane;
                const int e = min(max(at.r.len - w0, 0), 32), f = min(max(at.r.lo - w0, 0), 32);
                uint32_t m = (e == 32 ? 0xffffffffu : (1u << e) - 1u) & ~(f == 32 ? 0xffffffffu : (1u << f) - 1u);
                const uint32_t pg = ids >> ((32 * lane) >> sh);
                m &= page >= 32 ? ((pg & 1u) ? 0xffffffffu : 0u)
                                : ((pg & 1u) ? 0xffffu : 0u) | ((pg & 2u) ? 0xffff0000u : 0u);
                live_bits[s][lane] = m;
            }
            // codes: bulk copies, whole multiples of 4 tokens (16 bytes and more)
            const int ntok = min(page, (at.r.len - pt + 3) & ~3);
            const uint32_t bytes = has && id >= 0 ? static_cast<uint32_t>(ntok) * (D / 2) : 0u;
            const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full_bar[s], sum);
            __syncwarp();
            if (bytes > 0)
                bulk_load(ka_smem + s * L::kStage + dst0,
                          (vals ? p.c.vc : p.c.kc) + ((static_cast<int64_t>(id) * p.c.heads + at.kvh) * page) * (D / 2), bytes,
                          &full_bar[s]);
            // steps: 16-byte copies by every lane, whatever the page size (a bulk copy of a 16-token page's 64 or
            // 128 bytes would cost as much as one of its codes)
#pragma unroll
            for (int i = 0; i < L::kSteps / 512; ++i) {
                const int token = (lane + 32 * i) * (16 / (D / 16));
                const int from = __shfl_sync(0xffffffffu, id, token >> sh);
                if (from >= 0) {
                    const int64_t src = ((static_cast<int64_t>(from) * p.c.heads + at.kvh) * page + (token & (page - 1))) * (D / 32);
                    const uint32_t dst = ring + s * L::kStage + 2 * L::kCodes + 16u * (lane + 32 * i);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(p.c.ks + src) : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst + L::kSteps), "l"(p.c.vs + src) : "memory");
                }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(&full_bar[s])) : "memory");
            issued = u - u0 + 1;
            if (++s == kStages) { s = 0; ph ^= 1u; }
            at = ahead;
            id = id_next;
        }
        // no copy may still be landing when the CTA exits
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (lane == 0)
            for (int64_t i = (issued > kStages ? issued - kStages : 0); i < issued; ++i)
                mbar_wait(&full_bar[i % kStages], static_cast<uint32_t>(i / kStages) & 1u, nullptr, kDrainLimitNs);
        __syncwarp();
    } else {
        // ---------------------------------------------------------- consumers
        const int g = lane >> 2, t = lane & 3;
        const float c = p.scale_log2;
        uint32_t qb[kQs ? 1 : kN][2 * kW][2];       // q of row 8n + g, this thread's channels, operand order
        const uint32_t qs = ring + kStages * L::kStage + L::kJoin + 8u * lane;     // the same in shared memory
        float acc[kM][kN][4];
        float m[kN][2], l[kN][2];                   // of rows 8n + 2t and 8n + 2t + 1: reference maximum, sum
        int lim[kN][2], low[kN][2];                 // these rows see the tokens low..lim
        bool fresh = true, dead = false;
        bool rest = false;                          // the tile's sums before a fold are in its piece
        int seg = 0, seg_c0 = at.ch;
        int s = 0;
        uint32_t ph = 0;
        float* const join = reinterpret_cast<float*>(ka_smem + kStages * L::kStage);

        for (int64_t u = u0; u < u1; ++u) {
            if (fresh) {
                // a new tile: its queries in operand order, empty statistics
                const int rows = at.r.nq * p.group;
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const int row = at.tile * ROWS + 8 * n + g;
                    const bool in = row < rows && (!kLo || g < 4);
                    const int tok = in ? row / p.group : 0;
                    const uint16_t* src = p.q + (at.r.q0 + tok) * p.q_stride +
                                          static_cast<int64_t>(at.kvh * p.group + (in ? row - tok * p.group : 0)) * D + 8 * kW * t;
#pragma unroll
                    for (int w = 0; w < kW; ++w) {
                        if (kQs && (n * kW + w) % kKaWarps != warp) continue;        // the warps share this work
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (in) x = kv4_ld(reinterpret_cast<const uint4*>(src) + w);
                        const uint32_t y[4] = {__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                                               __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632)};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (kQs) {
                                asm volatile("st.shared.v2.b32 [%0], {%1, %2};"
                                             :: "r"(qs + 256u * (n * 2 * kW + 2 * w + i)), "r"(y[2 * i]), "r"(y[2 * i + 1]) : "memory");
                            } else {
                                qb[kQs ? 0 : n][2 * w + i][0] = y[2 * i];
                                qb[kQs ? 0 : n][2 * w + i][1] = y[2 * i + 1];
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int rr = at.tile * ROWS + 8 * n + 2 * t + e;
                        const bool there = rr < rows && (!kLo || t < 2);
                        const int pos = at.r.first + (there ? rr / p.group : 0);
                        // rows that do not exist see everything: their zero queries are harmless, and masks stay rare
                        lim[n][e] = !there ? 0x7fffffff : p.causal ? pos : at.r.len - 1;
                        low[n][e] = there && p.window > 0 ? pos - p.window + 1 : 0;
                        m[n][e] = -INFINITY;
                        l[n][e] = 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < kM; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][n][j] = 0.0f;
                }
                if (kQs) asm volatile("bar.sync 1, %0;" :: "n"(32 * kKaWarps) : "memory");
                if (!FOLD || !rest) seg_c0 = at.ch;
                fresh = false;
            }
            dead = dead || !kv4_wait(&full_bar[s], ph, abort, p.limit_ns);
            dead = __any_sync(0xffffffffu, dead);
            if (!dead) {
                const uint32_t sb = ring + s * L::kStage;
                const uint32_t live = live_bits[s][warp];
                const int t0 = at.t0() + 32 * warp;                  // first token of this warp's 32
                // 32 tokens at once, 16 where registers run out
#pragma unroll 1
                for (int k0 = 0; k0 < 2; k0 += kPass) {
                // ---- S^T = K Q^T, tiles of 16 tokens
                float sv[kPass][kN][4];
                const uint32_t kbase = sb + (32 * warp + g) * (D / 2) + 4 * kW * t;
                const uint32_t sbase = sb + 2 * L::kCodes + (32 * warp + g) * (D / 32) * 2 + 2 * (t * kW / 4);
#pragma unroll
                for (int k = 0; k < kPass; ++k) {
                    uint32_t w[2][kW], s2[2];                 // tokens g and g + 8 of the tile
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (kW == 4) {
                            const uint4 x = gm_lds128(kbase + (16 * (k0 + k) + 8 * h) * (D / 2));
                            w[h][0] = x.x; w[h][1] = x.y; w[h][2 % kW] = x.z; w[h][3 % kW] = x.w;
                        } else {
                            const uint2 x = lds64(kbase + (16 * (k0 + k) + 8 * h) * (D / 2));
                            w[h][0] = x.x; w[h][1] = x.y;
                        }
                        s2[h] = __byte_perm(lds_u16(sbase + (16 * (k0 + k) + 8 * h) * (D / 32) * 2), 0u, 0x1010);
                    }
#pragma unroll
                    for (int i = 0; i < kW; ++i) {
                        uint32_t a[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            a[0][h] = kv4_pair<0>(w[h][i], s2[h]);
                            a[0][2 + h] = kv4_pair<1>(w[h][i], s2[h]);
                            a[1][h] = kv4_pair<2>(w[h][i], s2[h]);
                            a[1][2 + h] = kv4_pair<3>(w[h][i], s2[h]);
                        }
#pragma unroll
                        for (int n = 0; n < kN; ++n) {
                            uint2 q0, q1;
                            if (kQs) {
                                q0 = lds64(qs + 256u * (n * 2 * kW + 2 * i));
                                q1 = lds64(qs + 256u * (n * 2 * kW + 2 * i + 1));
                            } else {
                                const uint32_t (&y)[2 * kW][2] = qb[kQs ? 0 : n];
                                q0 = make_uint2(y[2 * i][0], y[2 * i][1]);
                                q1 = make_uint2(y[2 * i + 1][0], y[2 * i + 1][1]);
                            }
                            if (i == 0) ka_mma0(sv[k][n], a[0][0], a[0][1], a[0][2], a[0][3], q0.x, q0.y);
                            else gm_mma(sv[k][n], a[0][0], a[0][1], a[0][2], a[0][3], q0.x, q0.y);
                            gm_mma(sv[k][n], a[1][0], a[1][1], a[1][2], a[1][3], q1.x, q1.y);
                        }
                    }
                }
                // ---- masks: tokens that do not exist, and each row's own range
                bool plain = live == 0xffffffffu;
#pragma unroll
                for (int n = 0; n < kN; ++n)
                    plain = plain && min(lim[n][0], lim[n][1]) >= t0 + 31 && max(low[n][0], low[n][1]) <= t0;
                if (!__all_sync(0xffffffffu, plain)) {
#pragma unroll
                    for (int k = 0; k < kPass; ++k)
#pragma unroll
                        for (int n = 0; n < kN; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int off = 16 * (k0 + k) + g + 8 * (i >> 1), tk = t0 + off;
                                if (!((live >> off) & 1u) || tk > lim[n][i & 1] || tk < low[n][i & 1]) sv[k][n][i] = -INFINITY;
                            }
                }
                // ---- reference maxima move, and outputs are rescaled, only when a score exceeds them by 2^kKaGrow
                float x[kN][2];
                bool grow = false;
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float y = fmaxf(sv[0][n][e], sv[0][n][2 + e]);
                        if (kPass == 2) y = fmaxf(y, fmaxf(sv[kPass - 1][n][e], sv[kPass - 1][n][2 + e]));
                        x[n][e] = y * c;
                        grow = grow || x[n][e] > m[n][e] + kKaGrow;
                    }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float y = x[n][e];
#pragma unroll
                            for (int d = 4; d <= 16; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                            const bool up = y > m[n][e] + kKaGrow;      // the same in the row's 8 lanes
                            float a = up ? ex2(m[n][e] - y) : 1.0f;
                            if (up) m[n][e] = y;
                            l[n][e] *= a;
                            if (kLo) {                                  // the remainders' columns go with their rows
                                const float b = __shfl_xor_sync(0xffffffffu, a, 2);
                                if (t >= 2) a = b;
                            }
#pragma unroll
                            for (int i = 0; i < kM; ++i) {
                                acc[i][n][e] *= a;
                                acc[i][n][2 + e] *= a;
                            }
                        }
                }
                // ---- P, transposed into the second product's operand
                uint32_t pb[kPass][kN][2];
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const float n0 = m[n][0] == -INFINITY ? 0.0f : -m[n][0], n1 = m[n][1] == -INFINITY ? 0.0f : -m[n][1];
#pragma unroll
                    for (int k = 0; k < kPass; ++k)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float e0 = ex2(fmaf(sv[k][n][2 * h], c, n0)), e1 = ex2(fmaf(sv[k][n][2 * h + 1], c, n1));
                            l[n][0] += e0;
                            l[n][1] += e1;
                            uint32_t hi = pack_bf16(e0, e1);
                            if (kLo) {
                                const uint32_t lo = __shfl_xor_sync(
                                    0xffffffffu, pack_bf16(e0 - __uint_as_float(hi << 16), e1 - __uint_as_float(hi & 0xFFFF0000u)), 2);
                                if (t >= 2) hi = lo;
                            }
                            pb[k][n][h] = ka_trans(hi);
                        }
                }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int k = 0; k < kPass; ++k) {
                    uint32_t v[2][8 * kVW];                  // pairs of tokens (2t, 2t+1) and (2t+8, 2t+9)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int off = 16 * (k0 + k) + 8 * h + 2 * t;
                        const uint32_t vb = sb + L::kCodes + (32 * warp + off) * (D / 2) + 4 * kVW * g;
                        const uint32_t ss = sb + 2 * L::kCodes + L::kSteps + (32 * warp + off) * (D / 32) * 2 + 2 * (kVW * g / 4);
                        uint32_t wa[kVW], wb[kVW];
                        if (kVW == 2) {
                            const uint2 xa = lds64(vb), xb = lds64(vb + D / 2);
                            wa[0] = xa.x; wa[1 % kVW] = xa.y;
                            wb[0] = xb.x; wb[1 % kVW] = xb.y;
                        } else {
                            wa[0] = gm_lds32(vb);
                            wb[0] = gm_lds32(vb + D / 2);
                        }
                        uint32_t s2 = __byte_perm(lds_u16(ss), lds_u16(ss + (D / 32) * 2), 0x5410);
                        if (live != 0xffffffffu)               // tokens that do not exist: step 0
                            s2 &= (((live >> off) & 1u) ? 0xffffu : 0u) | (((live >> (off + 1)) & 1u) ? 0xffff0000u : 0u);
#pragma unroll
                        for (int i = 0; i < kVW; ++i) {
                            const uint32_t lo = __byte_perm(wa[i], wb[i], 0x5410), hi = __byte_perm(wa[i], wb[i], 0x7632);
                            v[h][8 * i + 0] = kv4_pair<0>(lo, s2);
                            v[h][8 * i + 1] = kv4_pair<1>(lo, s2);
                            v[h][8 * i + 2] = kv4_pair<2>(lo, s2);
                            v[h][8 * i + 3] = kv4_pair<3>(lo, s2);
                            v[h][8 * i + 4] = kv4_pair<0>(hi, s2);
                            v[h][8 * i + 5] = kv4_pair<1>(hi, s2);
                            v[h][8 * i + 6] = kv4_pair<2>(hi, s2);
                            v[h][8 * i + 7] = kv4_pair<3>(hi, s2);
                        }
                    }
                    // rows g and g + 8 of tile i: this thread's channels i and i + kM
#pragma unroll
                    for (int i = 0; i < kM; ++i)
#pragma unroll
                        for (int n = 0; n < kN; ++n)
                            gm_mma(acc[i][n], v[0][i], v[0][kM + i], v[1][i], v[1][kM + i], pb[k][n][0], pb[k][n][1]);
                }
                }
            }
            // the slot is released only once what was loaded from it has been used
            __syncwarp();
            if (lane == 0 && !dead) mbar_arrive(&empty_bar[s]);
            if (++s == kStages) { s = 0; ph ^= 1u; }

            const bool tile_end = at.ch == at.un.chunks - 1;
            const bool last = tile_end || u == u1 - 1;
            if (last || (FOLD && ((at.ch - seg_c0) & (kKaFold - 1)) == kKaFold - 1)) {
                // ---- join the four warps, then write the rows or leave the piece to be joined with others
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int d = 4; d <= 16; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
                        if (g == 0 && (!kLo || t < 2)) {
                            join_m[warp][8 * n + 2 * t + e] = m[n][e];
                            join_l[warp][8 * n + 2 * t + e] = l[n][e];
                        }
                        float o[2 * kM];                      // the row's channels 2 kM g ..
#pragma unroll
                        for (int i = 0; i < kM; ++i) {
                            o[i] = acc[i][n][e];
                            o[kM + i] = acc[i][n][2 + e];
                        }
                        if (kLo) {
#pragma unroll
                            for (int i = 0; i < 2 * kM; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], 2);
                        }
                        if (!kLo || t < 2) {
                            float4* dst = reinterpret_cast<float4*>(join + (warp * ROWS + 8 * n + 2 * t + e) * (L::kORow / 4) + 2 * kM * g);
#pragma unroll
                            for (int i = 0; i < kM / 2; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                    }
                asm volatile("bar.sync 1, %0;" :: "n"(32 * kKaWarps) : "memory");
                const int rows = at.r.nq * p.group - at.tile * ROWS;     // rows of this tile that exist
                const bool whole = !CL && seg_c0 == 0 && tile_end;      // no other CTA has keys of this tile
                const int slot = 2 * static_cast<int>(blockIdx.x) + (seg > 0 ? 1 : 0);
                float* const piece = CL ? res : p.part + static_cast<int64_t>(slot) * ka_piece<D, ROWS>();
                constexpr int kPer = D / 8;                             // threads per row: 8 channels each
                for (int x = tid; x < ROWS * kPer; x += 32 * kKaWarps) {
                    const int row = x / kPer, d0 = (x - row * kPer) * 8;
                    if (row >= rows) break;
                    float mm = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kKaWarps; ++w) mm = fmaxf(mm, join_m[w][row]);
                    float ll = 0.0f, o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < kKaWarps; ++w) {
                        const float f = mm == -INFINITY ? 0.0f : ex2(join_m[w][row] - mm);
                        ll += f * join_l[w][row];
                        const float4* src = reinterpret_cast<const float4*>(join + (w * ROWS + row) * (L::kORow / 4) + d0);
                        const float4 a = src[0], e = src[1];
                        o[0] += f * a.x; o[1] += f * a.y; o[2] += f * a.z; o[3] += f * a.w;
                        o[4] += f * e.x; o[5] += f * e.y; o[6] += f * e.z; o[7] += f * e.w;
                    }
                    if (FOLD && rest) {
                        // what an earlier fold left; the row's threads, lanes of one warp, read before one writes
                        const float m0 = piece[ROWS * D + row], l0 = piece[ROWS * D + ROWS + row];
                        const float4* src = reinterpret_cast<const float4*>(piece + row * D + d0);
                        const float4 a = src[0], e = src[1];
                        __syncwarp(((1u << kPer) - 1u) << (lane & ~(kPer - 1)));
                        const float top = fmaxf(mm, m0);
                        const float f = top == -INFINITY ? 0.0f : ex2(mm - top), f0 = top == -INFINITY ? 0.0f : ex2(m0 - top);
                        mm = top;
                        ll = f * ll + f0 * l0;
                        o[0] = f * o[0] + f0 * a.x; o[1] = f * o[1] + f0 * a.y; o[2] = f * o[2] + f0 * a.z; o[3] = f * o[3] + f0 * a.w;
                        o[4] = f * o[4] + f0 * e.x; o[5] = f * o[5] + f0 * e.y; o[6] = f * o[6] + f0 * e.z; o[7] = f * o[7] + f0 * e.w;
                    }
                    if (*abort) continue;
                    if (whole) {
                        const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
                        const int64_t to = ka_out_row(p, at.r, at.kvh, at.tile * ROWS + row);
                        *reinterpret_cast<uint4*>(p.out + to * D + d0) =
                            make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                                       pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
                        if (d0 == 0 && p.lse) p.lse[to] = kv4_lse(mm, ll);
                    } else {
                        float4* dst = reinterpret_cast<float4*>(piece + row * D + d0);
                        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                        if (d0 == 0) {
                            piece[ROWS * D + row] = mm;
                            piece[ROWS * D + ROWS + row] = ll;
                        }
                    }
                }
                if (!CL && last && !whole && tid == 0)
                    p.meta[2 * blockIdx.x + (seg > 0 ? 1 : 0)] =
                        make_int4(at.b, at.kvh * at.un.tiles + at.tile, seg_c0, tile_end ? -(at.ch + 1) : at.ch + 1);
                asm volatile("bar.sync 1, %0;" :: "n"(32 * kKaWarps) : "memory");
                fresh = true;
                rest = !last;
                if (last) ++seg;
            }
            if (u + 1 < u1) at.next(p, true);
        }
        if (CL && u0 >= u1) {
            // no chunk for this CTA: an empty piece
            for (int x = tid; x < ka_piece<D, ROWS>(); x += 32 * kKaWarps)
                res[x] = x >= ROWS * D && x < ROWS * D + ROWS ? -INFINITY : 0.0f;
        }
    }
    if (CL) {
        // ---- the cluster's pieces joined: each CTA takes its share of (row, 4 channels)
        __syncwarp();
        cluster_sync_all();
        const int rank = static_cast<int>(cluster_ctarank());
        // the place of the tile (the roles above may have moved on)
        const Request r = kv4_request(p, s_b);
        const Units<ROWS> un = kv4_units<ROWS>(p, r);
        const int kvh = static_cast<int>(s_skip / un.tiles), tile = static_cast<int>(s_skip % un.tiles);
        const int rows = r.nq * p.group - tile * ROWS;
        constexpr int kPer = D / 4, kShare = ROWS * kPer / kKaCluster;
        const int x = rank * kShare + tid, row = x / kPer, d0 = (x - row * kPer) * 4;
        if (tid < kShare && row < rows && !*abort) {
            uint32_t from[kKaCluster];
            float mj[kKaCluster], mm = -INFINITY;
#pragma unroll
            for (int j = 0; j < kKaCluster; ++j) {
                from[j] = cluster_map(res, j);
                mj[j] = ld_cluster_f32(from[j] + (ROWS * D + row) * 4);
            }
#pragma unroll
            for (int j = 0; j < kKaCluster; ++j) mm = fmaxf(mm, mj[j]);
            float ll = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < kKaCluster; ++j) {
                const float f = mm == -INFINITY ? 0.0f : ex2(mj[j] - mm);
                const float4 v = ld_cluster_f32x4(from[j] + (row * D + d0) * 4);
                ll += f * ld_cluster_f32(from[j] + (ROWS * D + ROWS + row) * 4);
                o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
            }
            const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
            const int64_t to = ka_out_row(p, r, kvh, tile * ROWS + row);
            *reinterpret_cast<uint2*>(p.out + to * D + d0) =
                make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
            if (d0 == 0 && p.lse) p.lse[to] = kv4_lse(mm, ll);
        }
        __syncwarp();
        cluster_sync_all();      // no CTA leaves while another may still read its piece
    }
}

// Joins the pieces of a cut tile.  Records: (request, kvh * tiles + tile, first chunk, end chunk --
// negated when the tile ends there), first word -1 where the CTA left no piece.  The block of the
// CTA that holds a tile's first piece owns it; the following pieces are the first records of the
// next CTAs, up to the one that ends the tile.  Four rows per block (blockIdx.y), two warps per row
// that take every other piece, eight of them in flight (a request over the whole GPU has dozens: one of
// 131,071 tokens took 50 us with both kernels, 60 with one piece in flight).
constexpr int kKcThreads = 256;
template <int D, int ROWS>
__global__ void __launch_bounds__(kKcThreads)
kv4_combine_kernel(const AttnParams p, int ctas) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int s_end;
    __shared__ float part[4][D + 2];       // what a row's second warp found
    const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int4 a = p.meta[2 * c], e = p.meta[2 * c + 1];
    int slot = -1;
    int4 me = a;
    if (a.x >= 0 && a.z == 0 && a.w > 0) slot = 2 * c;
    if (e.x >= 0 && e.z == 0 && e.w > 0) { slot = 2 * c + 1; me = e; }
    if (slot < 0) return;
    const Request r = kv4_request(p, me.x);
    const Units<ROWS> un = kv4_units<ROWS>(p, r);
    const int tile = me.y % un.tiles, kvh = me.y / un.tiles;
    if (tid == 0) s_end = ctas;
    __syncthreads();
    // the piece that ends the tile: the first of the following CTAs' first records with a negated end
    for (int j = c + 1 + tid; j < ctas; j += kKcThreads) {
        const int4 m = p.meta[2 * j];
        const bool same = m.x == me.x && m.y == me.y;
        if (!same) atomicMin(&s_end, j);
        else if (m.w < 0) atomicMin(&s_end, j + 1);
    }
    __syncthreads();
    const int pieces = s_end - c;                                 // slot, then 2j for c < j < s_end
    const int q = tid >> 6, half = (tid >> 5) & 1;                // row of this block's four, every other piece
    const int row = 4 * blockIdx.y + q;
    const int rows = min(ROWS, r.nq * p.group - tile * ROWS);
    constexpr int n = ka_piece<D, ROWS>();
    constexpr int kC = D / 32;                                    // channels per lane
    float mm = -INFINITY, ll = 0.0f, o[kC] = {};
    if (row < rows) {
        for (int j0 = half; j0 < pieces; j0 += 16) {
            float mj[8], lj[8], v[8][kC];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = j0 + 2 * i;
                const float* src = p.part + static_cast<int64_t>(j == 0 ? slot : 2 * (c + j)) * n;
                const bool in = j < pieces;
                mj[i] = in ? src[ROWS * D + row] : -INFINITY;
                lj[i] = in ? src[ROWS * D + ROWS + row] : 0.0f;
#pragma unroll
                for (int k = 0; k < kC; k += 2) {
                    const float2 x = in ? *reinterpret_cast<const float2*>(src + row * D + kC * lane + k) : make_float2(0.0f, 0.0f);
                    v[i][k] = x.x;
                    v[i][k + 1] = x.y;
                }
            }
            float top = mm;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, mj[i]);
            const float f0 = top == -INFINITY ? 0.0f : ex2(mm - top);
            mm = top;
            ll *= f0;
#pragma unroll
            for (int k = 0; k < kC; ++k) o[k] *= f0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = top == -INFINITY ? 0.0f : ex2(mj[i] - top);
                ll += f * lj[i];
#pragma unroll
                for (int k = 0; k < kC; ++k) o[k] += f * v[i][k];
            }
        }
        if (half == 1) {
#pragma unroll
            for (int k = 0; k < kC; ++k) part[q][kC * lane + k] = o[k];
            if (lane == 0) { part[q][D] = mm; part[q][D + 1] = ll; }
        }
    }
    __syncthreads();
    if (row >= rows || half == 1) return;
    const float m1 = part[q][D], top = fmaxf(mm, m1);
    const float f0 = top == -INFINITY ? 0.0f : ex2(mm - top), f1 = top == -INFINITY ? 0.0f : ex2(m1 - top);
    ll = ll * f0 + part[q][D + 1] * f1;
    const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
    const int64_t at = ka_out_row(p, r, kvh, tile * ROWS + row);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * D + kC * lane);
#pragma unroll
    for (int k = 0; k < kC; k += 2)
        dst[k / 2] = pack_bf16((o[k] * f0 + part[q][kC * lane + k] * f1) * inv,
                               (o[k + 1] * f0 + part[q][kC * lane + k + 1] * f1) * inv);
    if (lane == 0 && p.lse) p.lse[at] = kv4_lse(top, ll);
}

}  // namespace qat4
