// kv4_attn.cuh -- softmax attention of a ragged batch of queries over the
// paged 4-bit cache (kv4_cache.cuh), for few query rows per request: decode
// steps and short drafts.
//     o_i = sum_j softmax_j(scale q_i . k_j) v_j  over the keys j that query i
//     may see (j <= pos_i when causal, j > pos_i - window when windowed)
//
// Rows.  The group = q_heads / kv_heads query heads that share a key/value head
// are packed with the request's query tokens into rows (token * group + head),
// so a cached token is read once for all of them: a tile is ROWS = 8 or 16 rows
// of the 16 of an mma.sync m16n8k16 (with 8, the accumulators and exponentials
// of the upper half are left out).
//
// Bound: HBM.  A cached token of a head costs 2 * (D/2 + D/16) bytes (144 at
// D = 128) and 4 * D * rows flop, far below the tensor cores' balance, so the
// contractions run on mma.sync only to keep the issue slots for the decoding:
// per pair of codes one shift, one logic op and one packed FMA (kv4_pair).  The
// operand orders are chosen so that the packed words need no reordering:
//   S = Q K^T: B = keys.  Thread (g, t) holds token g of an 8-token tile and its
//     channels [32t, 32t + 32) (D = 128): 16 bytes of codes and one step; the
//     8 MMAs of a tile take word w's pairs (0,4)(1,5) and (2,6)(3,7), and q is
//     loaded once in that order.
//   O = P V: B = values.  Thread (g, t) holds channels [16g, 16g + 16) of the
//     tokens (2t, 2t+1), (2t+8, 2t+9); a byte permute pairs two tokens' words
//     and the same decode gives the (token, token + 1) pairs of each channel.
//     The accumulator columns of thread t are then 32 consecutive channels.
// P is the accumulator of S rounded to bf16 (half a step, 2^-9 of each weight;
// the row sum adds the unrounded weights), the statistics are float32.
//
// Work split.  A unit is (request, kv head, row tile, chunk of 128 tokens); the
// units of the whole ragged batch form one list (from the lengths, on the
// device) that is cut into equal ranges, one per CTA, so a long request spreads
// over the GPU and a batch of ragged ones leaves no CTA idle.  A tile cut
// between CTAs leaves (max, sum, unnormalised output) of each piece in the
// workspace, and kv4_combine_kernel joins them in order (no atomics: the result
// does not depend on timing).
//
// Data movement.  A producer warp streams each unit's pages with untiled bulk
// copies into a ring (one copy per page and array: a page's head is contiguous)
// and writes which of the 128 tokens exist: tokens past the length, of pages
// that the table does not name, or that no query of the request can see any
// more are never attended to, and their steps are taken as 0, whatever bytes
// lie there.  Four consumer warps take 32 tokens each with statistics of their
// own, joined at the end of a tile's piece.
#pragma once

#include <cuda_bf16.h>

#include "device_common.cuh"
#include "kv4_cache.cuh"
#include "w4a16_gemv.cuh"

namespace qat4 {

constexpr int kKaWarps = 4;                       // consumer warps
constexpr int kKaThreads = 32 * (kKaWarps + 1);   // + one producer warp
constexpr int kKaChunk = 128;                     // tokens per unit
constexpr int kKaStages = 4;
constexpr float kKaGrow = 8.0f;   // a row's reference maximum moves only when exceeded by 2^8

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
    const int a = min(max(__ldg(p.cu_q + b), 0), p.N), e = min(max(__ldg(p.cu_q + b + 1), 0), p.N);
    r.q0 = a;
    r.nq = max(0, e - a);
    const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.c.page;
    const int len = max(0, __ldg(p.seq_lens + b));
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

template <int D, int ROWS>
struct KaLayout {
    static constexpr int kCodes = kKaChunk * D / 2;
    static constexpr int kSteps = kKaChunk * (D / 32) * 2;
    static constexpr int kStage = 2 * kCodes + 2 * kSteps;
    static constexpr int kORow = D * 4 + 16;                      // bytes of an output row in the join buffer
    static constexpr int kJoin = kKaWarps * ROWS * kORow;
    static constexpr size_t kSmem = static_cast<size_t>(kKaStages) * kStage + kJoin;
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

// Row `row` of a tile's result: out (and lse) from the unnormalised sums.
__device__ __forceinline__ int64_t ka_out_row(const AttnParams& p, const Request& r, int kvh, int row) {
    const int tok = row / p.group;
    return static_cast<int64_t>(r.q0 + tok) * p.Hq + kvh * p.group + (row - tok * p.group);
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kKaThreads, 2)
kv4_decode_kernel(const AttnParams p) {
    using L = KaLayout<D, ROWS>;
    constexpr bool kFull = ROWS == 16;
    constexpr int kSteps = D / 16;             // MMAs along the channels of S
    constexpr int kW = D / 32;                 // words of a thread's key channels (4 or 2)
    constexpr int kVW = D / 64;                // words of a thread's value channels (2 or 1)
    constexpr int kNT = D / 8;                 // output tiles of 8 channels
    extern __shared__ __align__(128) uint8_t ka_smem[];
    __shared__ __align__(8) uint64_t full_bar[kKaStages], empty_bar[kKaStages];
    __shared__ uint32_t live_bits[kKaStages][4];
    __shared__ float join_m[kKaWarps][16], join_l[kKaWarps][16];
    __shared__ int64_t scan[32], s_skip;
    __shared__ int s_b;
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();

    // ---- this CTA's range of the unit list
    const int per = (p.B + kKaThreads - 1) / kKaThreads;
    const int rb0 = min(p.B, tid * per), rb1 = min(p.B, rb0 + per);
    int64_t mine = 0;
    for (int b = rb0; b < rb1; ++b) {
        const Request r = kv4_request(p, b);
        const Units<ROWS> u = kv4_units<ROWS>(p, r);
        mine += static_cast<int64_t>(u.tiles) * u.chunks * p.c.heads;
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += a;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) {
        s_b = p.B;
        abort_flag = 0;
        for (int s = 0; s < kKaStages; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], kKaWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int w = 0; w <= kKaWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);     // every CTA of these has work
    const int64_t u0 = ctas > 0 && blockIdx.x < ctas ? total * blockIdx.x / ctas : 0;
    const int64_t u1 = ctas > 0 && blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : 0;
    if (u0 < u1 && u0 >= before && u0 < before + mine) {
        int64_t at = before;
        for (int b = rb0; b < rb1; ++b) {
            const Request r = kv4_request(p, b);
            const Units<ROWS> u = kv4_units<ROWS>(p, r);
            const int64_t n = static_cast<int64_t>(u.tiles) * u.chunks * p.c.heads;
            if (u0 < at + n) {
                s_b = b;
                s_skip = u0 - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    int4* const meta = p.meta + 2 * blockIdx.x;
    if (tid < 2) meta[tid] = make_int4(-1, 0, 0, 0);
    if (u0 >= u1) return;
    __syncthreads();                            // the records below overwrite these
    volatile int* abort = &abort_flag;
    const int b_first = s_b;
    const int64_t skip = s_skip;
    const uint32_t ring = smem_u32(ka_smem);

    // position in the list: request b, kv head, tile and chunk of unit u0
    Request r = kv4_request(p, b_first);
    Units<ROWS> un = kv4_units<ROWS>(p, r);
    int b = b_first;
    int ch = static_cast<int>(skip % un.chunks);
    int tile = static_cast<int>((skip / un.chunks) % un.tiles);
    int kvh = static_cast<int>(skip / (static_cast<int64_t>(un.chunks) * un.tiles));
    const int page = p.c.page, sh = __ffs(page) - 1;

    if (warp == kKaWarps) {
        // ------------------------------------------------------------ producer
        const int np = kKaChunk >> sh;                         // pages per chunk, 1..8
        const int arr = lane / np, pi = lane - arr * np;       // lane's array and page
        const bool has = lane < 4 * np;
        const int unit = (arr & 1) ? (D / 32) * 2 : D / 2;     // bytes per token of the array
        const uint8_t* base = arr == 0 ? p.c.kc : arr == 1 ? reinterpret_cast<const uint8_t*>(p.c.ks)
                            : arr == 2 ? p.c.vc : reinterpret_cast<const uint8_t*>(p.c.vs);
        const uint32_t dst0 = (arr == 0 ? 0 : arr == 1 ? 2 * L::kCodes : arr == 2 ? L::kCodes : 2 * L::kCodes + L::kSteps) +
                              pi * page * unit;
        int64_t issued = 0;
        int s = 0;
        uint32_t ph = 0;
        for (int64_t u = u0; u < u1; ++u) {
            int ok = 1;
            if (lane == 0) ok = mbar_wait(&empty_bar[s], ph ^ 1u, abort, p.limit_ns) ? 1 : 0;
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            const int t0 = (un.c0 + ch) * kKaChunk;            // first token of the chunk
            const int pt = t0 + pi * page;                     // first token of this lane's page
            int id = -1;
            if (has && pt < r.len && pt + page > r.lo) {       // pt < len keeps the index inside the table's row
                id = __ldg(p.table + b * p.table_stride + (pt >> sh));
                if (id < 0 || id >= p.c.pages) id = -1;
            }
            // tokens that exist, 32 per word: lanes 0..3 take one word each from the pages' votes
            const uint32_t ids = __ballot_sync(0xffffffffu, has && arr == 0 && id >= 0);
            if (lane < 4) {
                uint32_t m = 0;
#pragma unroll 8
                for (int j = 0; j < 32; ++j) {
                    const int t = t0 + 32 * lane + j;
                    if (t < r.len && t >= r.lo && ((ids >> ((t - t0) >> sh)) & 1u)) m |= 1u << j;
                }
                live_bits[s][lane] = m;
            }
            // whole multiples of 4 tokens, so that every copy is a multiple of 16 bytes
            const int ntok = min(page, (r.len - pt + 3) & ~3);
            const uint32_t bytes = id >= 0 ? static_cast<uint32_t>(ntok * unit) : 0u;
            const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full_bar[s], sum);
            __syncwarp();
            if (bytes > 0)
                bulk_load(ka_smem + s * L::kStage + dst0,
                          base + ((static_cast<int64_t>(id) * p.c.heads + kvh) * page) * unit, bytes, &full_bar[s]);
            issued = u - u0 + 1;
            if (++s == kKaStages) { s = 0; ph ^= 1u; }
            if (++ch == un.chunks) {
                ch = 0;
                if (++tile == un.tiles) {
                    tile = 0;
                    if (++kvh == p.c.heads) {
                        kvh = 0;
                        if (u + 1 < u1) {
                            do {
                                ++b;
                                r = kv4_request(p, b);
                                un = kv4_units<ROWS>(p, r);
                            } while (un.tiles == 0);
                        }
                    }
                }
            }
        }
        // no copy may still be landing when the CTA exits
        if (lane == 0)
            for (int64_t i = (issued > kKaStages ? issued - kKaStages : 0); i < issued; ++i)
                mbar_wait(&full_bar[i % kKaStages], static_cast<uint32_t>(i / kKaStages) & 1u, nullptr, kDrainLimitNs);
        return;
    }

    // -------------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    const float c = p.scale_log2;
    uint32_t qa[kSteps][kFull ? 4 : 2];
    float acc[kNT][kFull ? 4 : 2];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    int lim0 = 0, lim1 = 0, low0 = 0, low1 = 0;     // rows g and g + 8 see the tokens low..lim
    bool fresh = true, dead = false;
    int seg = 0, seg_c0 = ch;
    int s = 0;
    uint32_t ph = 0;
    float* const join = reinterpret_cast<float*>(ka_smem + kKaStages * L::kStage);

    for (int64_t u = u0; u < u1; ++u) {
        if (fresh) {
            // a new tile: its queries in operand order, empty statistics
            const int rows = r.nq * p.group;
#pragma unroll
            for (int h = 0; h < (kFull ? 2 : 1); ++h) {
                const int row = tile * ROWS + g + 8 * h;
                const bool in = row < rows;
                const int tok = in ? row / p.group : 0;
                const uint16_t* src = p.q + (r.q0 + tok) * p.q_stride +
                                      static_cast<int64_t>(kvh * p.group + (in ? row - tok * p.group : 0)) * D + 8 * kW * t;
#pragma unroll
                for (int w = 0; w < kW; ++w) {
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (in) x = __ldg(reinterpret_cast<const uint4*>(src) + w);
                    qa[2 * w][h] = __byte_perm(x.x, x.z, 0x5410);
                    qa[2 * w][(kFull ? 2 : 1) + h] = __byte_perm(x.x, x.z, 0x7632);
                    qa[2 * w + 1][h] = __byte_perm(x.y, x.w, 0x5410);
                    qa[2 * w + 1][(kFull ? 2 : 1) + h] = __byte_perm(x.y, x.w, 0x7632);
                }
                const int pos = r.first + tok;
                // rows past the last query see everything: their zero queries are harmless, and masks stay rare
                const int lim = !in ? 0x7fffffff : p.causal ? pos : r.len - 1;
                const int low = in && p.window > 0 ? pos - p.window + 1 : 0;
                if (h == 0) { lim0 = lim; low0 = low; } else { lim1 = lim; low1 = low; }
            }
#pragma unroll
            for (int i = 0; i < kNT; ++i)
#pragma unroll
                for (int j = 0; j < (kFull ? 4 : 2); ++j) acc[i][j] = 0.0f;
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.0f;
            seg_c0 = ch;
            fresh = false;
        }
        dead = dead || !mbar_wait(&full_bar[s], ph, abort, p.limit_ns);
        dead = __any_sync(0xffffffffu, dead);
        if (!dead) {
            const uint32_t sb = ring + s * L::kStage;
            const uint32_t live = live_bits[s][warp];
            const int t0 = (un.c0 + ch) * kKaChunk + 32 * warp;       // first token of this warp's 32
            // ---- S = Q K^T
            float sv[4][kFull ? 4 : 2];
            const uint32_t kbase = sb + (32 * warp + g) * (D / 2) + 4 * kW * t;
            const uint32_t sbase = sb + 2 * L::kCodes + (32 * warp + g) * (D / 32) * 2 + 2 * (t * kW / 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[kW];
                if (kW == 4) {
                    const uint4 x = gm_lds128(kbase + j * 8 * (D / 2));
                    w[0] = x.x; w[1] = x.y; w[2 % kW] = x.z; w[3 % kW] = x.w;
                } else {
                    const uint2 x = lds64(kbase + j * 8 * (D / 2));
                    w[0] = x.x; w[1] = x.y;
                }
                const uint32_t st = lds_u16(sbase + j * 8 * (D / 32) * 2);
                const uint32_t s2 = st | (st << 16), o2 = kv4_off(s2);
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    const uint32_t b0 = kv4_pair(w[i] << 3, s2, o2), b1 = kv4_pair(w[i] >> 1, s2, o2);
                    const uint32_t b2 = kv4_pair(w[i] >> 5, s2, o2), b3 = kv4_pair(w[i] >> 9, s2, o2);
                    if (kFull) {
                        gm_mma(d, qa[2 * i][0], qa[2 * i][1], qa[2 * i][2 % (kFull ? 4 : 2)], qa[2 * i][3 % (kFull ? 4 : 2)], b0, b1);
                        gm_mma(d, qa[2 * i + 1][0], qa[2 * i + 1][1], qa[2 * i + 1][2 % (kFull ? 4 : 2)],
                               qa[2 * i + 1][3 % (kFull ? 4 : 2)], b2, b3);
                    } else {
                        gm_mma(d, qa[2 * i][0], 0u, qa[2 * i][1], 0u, b0, b1);
                        gm_mma(d, qa[2 * i + 1][0], 0u, qa[2 * i + 1][1], 0u, b2, b3);
                    }
                }
#pragma unroll
                for (int i = 0; i < (kFull ? 4 : 2); ++i) sv[j][i] = d[i];
            }
            // ---- masks: tokens that do not exist, and each row's own range
            const int mn = kFull ? min(lim0, lim1) : lim0, mx = kFull ? max(low0, low1) : low0;
            const bool plain = live == 0xffffffffu && mn >= t0 + 31 && mx <= t0;
            if (!__all_sync(0xffffffffu, plain)) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int off = 8 * j + 2 * t + i, tk = t0 + off;
                        const bool in = (live >> off) & 1u;
                        if (!(in && tk <= lim0 && tk >= low0)) sv[j][i] = -INFINITY;
                        if (kFull && !(in && tk <= lim1 && tk >= low1)) sv[j][(2 + i) % (kFull ? 4 : 2)] = -INFINITY;
                    }
            }
            // ---- running maximum; outputs are rescaled only when it grows by more than 2^kKaGrow
            float x0 = fmaxf(fmaxf(fmaxf(sv[0][0], sv[0][1]), fmaxf(sv[1][0], sv[1][1])),
                             fmaxf(fmaxf(sv[2][0], sv[2][1]), fmaxf(sv[3][0], sv[3][1])));
            float x1 = -INFINITY;
            if (kFull) {
                constexpr int a = 2 % (kFull ? 4 : 2), e = 3 % (kFull ? 4 : 2);
                x1 = fmaxf(fmaxf(fmaxf(sv[0][a], sv[0][e]), fmaxf(sv[1][a], sv[1][e])),
                           fmaxf(fmaxf(sv[2][a], sv[2][e]), fmaxf(sv[3][a], sv[3][e])));
            }
#pragma unroll
            for (int d = 1; d <= 2; d <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
                if (kFull) x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
            }
            x0 *= c;
            if (kFull) x1 *= c;
            // m - x is NaN only for -inf - -inf: nothing seen yet, nothing to do
            const bool grow0 = x0 > m0 + kKaGrow, grow1 = kFull && x1 > m1 + kKaGrow;
            if (__any_sync(0xffffffffu, grow0 || grow1)) {
                const float a0 = grow0 ? ex2(m0 - x0) : 1.0f, a1 = grow1 ? ex2(m1 - x1) : 1.0f;
                if (grow0) m0 = x0;
                if (grow1) m1 = x1;
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int i = 0; i < kNT; ++i) {
                    acc[i][0] *= a0;
                    acc[i][1] *= a0;
                    if (kFull) {
                        acc[i][2 % (kFull ? 4 : 2)] *= a1;
                        acc[i][3 % (kFull ? 4 : 2)] *= a1;
                    }
                }
            }
            const float n0 = m0 == -INFINITY ? 0.0f : -m0, n1 = m1 == -INFINITY ? 0.0f : -m1;
            uint32_t pa[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e0 = ex2(fmaf(sv[j][0], c, n0)), e1 = ex2(fmaf(sv[j][1], c, n0));
                l0 += e0 + e1;
                pa[j >> 1][2 * (j & 1)] = pack_bf16(e0, e1);
                if (kFull) {
                    const float e2 = ex2(fmaf(sv[j][2 % (kFull ? 4 : 2)], c, n1));
                    const float e3 = ex2(fmaf(sv[j][3 % (kFull ? 4 : 2)], c, n1));
                    l1 += e2 + e3;
                    pa[j >> 1][2 * (j & 1) + 1] = pack_bf16(e2, e3);
                } else {
                    pa[j >> 1][2 * (j & 1) + 1] = 0u;
                }
            }
            // ---- O += P V
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t bp[2][8 * kVW];                     // pairs of tokens (2t, 2t+1) and (2t+8, 2t+9)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int off = 16 * k + 8 * h + 2 * t;
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
                    if (live != 0xffffffffu)                   // tokens that do not exist: step 0
                        s2 &= (((live >> off) & 1u) ? 0xffffu : 0u) | (((live >> (off + 1)) & 1u) ? 0xffff0000u : 0u);
                    const uint32_t o2 = kv4_off(s2);
#pragma unroll
                    for (int i = 0; i < kVW; ++i) {
                        const uint32_t lo = __byte_perm(wa[i], wb[i], 0x5410), hi = __byte_perm(wa[i], wb[i], 0x7632);
                        bp[h][8 * i + 0] = kv4_pair(lo << 3, s2, o2);
                        bp[h][8 * i + 1] = kv4_pair(lo >> 1, s2, o2);
                        bp[h][8 * i + 2] = kv4_pair(lo >> 5, s2, o2);
                        bp[h][8 * i + 3] = kv4_pair(lo >> 9, s2, o2);
                        bp[h][8 * i + 4] = kv4_pair(hi << 3, s2, o2);
                        bp[h][8 * i + 5] = kv4_pair(hi >> 1, s2, o2);
                        bp[h][8 * i + 6] = kv4_pair(hi >> 5, s2, o2);
                        bp[h][8 * i + 7] = kv4_pair(hi >> 9, s2, o2);
                    }
                }
#pragma unroll
                for (int i = 0; i < kNT; ++i) {
                    if constexpr (kFull) {
                        gm_mma(acc[i], pa[k][0], pa[k][1], pa[k][2], pa[k][3], bp[0][i], bp[1][i]);
                    } else {
                        float d[4] = {acc[i][0], acc[i][1], 0.0f, 0.0f};
                        gm_mma(d, pa[k][0], 0u, pa[k][2], 0u, bp[0][i], bp[1][i]);
                        acc[i][0] = d[0];
                        acc[i][1] = d[1];
                    }
                }
            }
        }
        // the slot is released only once what was loaded from it has been used
        __syncwarp();
        if (lane == 0 && !dead) mbar_arrive(&empty_bar[s]);
        if (++s == kKaStages) { s = 0; ph ^= 1u; }

        const bool tile_end = ch == un.chunks - 1;
        if (tile_end || u == u1 - 1) {
            // ---- join the four warps, then write the rows or leave the piece in the workspace
#pragma unroll
            for (int d = 1; d <= 2; d <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, d);
                if (kFull) l1 += __shfl_xor_sync(0xffffffffu, l1, d);
            }
            if (t == 0) {
                join_m[warp][g] = m0;
                join_l[warp][g] = l0;
                if (kFull) {
                    join_m[warp][g + 8] = m1;
                    join_l[warp][g + 8] = l1;
                }
            }
#pragma unroll
            for (int h = 0; h < (kFull ? 2 : 1); ++h) {
                float* o = join + (warp * ROWS + g + 8 * h) * (L::kORow / 4) + 16 * kVW * t;
#pragma unroll
                for (int cc = 0; cc < 2; ++cc)                 // accumulator column: channels +0.. or + 8 kVW..
#pragma unroll
                    for (int i = 0; i < 8 * kVW; i += 4)
                        *reinterpret_cast<float4*>(o + cc * 8 * kVW + i) =
                            make_float4(acc[i][(2 * h + cc) % (kFull ? 4 : 2)], acc[i + 1][(2 * h + cc) % (kFull ? 4 : 2)],
                                        acc[i + 2][(2 * h + cc) % (kFull ? 4 : 2)], acc[i + 3][(2 * h + cc) % (kFull ? 4 : 2)]);
            }
            asm volatile("bar.sync 1, %0;" :: "n"(32 * kKaWarps) : "memory");
            const int rows = r.nq * p.group - tile * ROWS;     // rows of this tile that exist
            const bool whole = seg_c0 == 0 && tile_end;
            const int slot = 2 * static_cast<int>(blockIdx.x) + (seg > 0 ? 1 : 0);
            float* const piece = p.part + static_cast<int64_t>(slot) * ka_piece<D, ROWS>();
            constexpr int kPer = D / 8;                         // threads per row: 8 channels each
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
                if (*abort) continue;
                if (whole) {
                    const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
                    const int64_t at = ka_out_row(p, r, kvh, tile * ROWS + row);
                    *reinterpret_cast<uint4*>(p.out + at * D + d0) =
                        make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                                   pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
                    if (d0 == 0 && p.lse) p.lse[at] = ll > 0.0f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
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
            if (!whole && tid == 0)
                meta[seg > 0 ? 1 : 0] = make_int4(b, kvh * un.tiles + tile, seg_c0, ch + 1 == un.chunks ? -(ch + 1) : ch + 1);
            asm volatile("bar.sync 1, %0;" :: "n"(32 * kKaWarps) : "memory");
            fresh = true;
            ++seg;
        }
        if (++ch == un.chunks) {
            ch = 0;
            if (++tile == un.tiles) {
                tile = 0;
                if (++kvh == p.c.heads) {
                    kvh = 0;
                    if (u + 1 < u1) {
                        do {
                            ++b;
                            r = kv4_request(p, b);
                            un = kv4_units<ROWS>(p, r);
                        } while (un.tiles == 0);
                    }
                }
            }
        }
    }
}

// Joins the pieces of a cut tile.  Records: (request, kvh * tiles + tile, first chunk, end chunk --
// negated when the tile ends there), first word -1 where the CTA left no piece.  The block of the
// CTA that holds a tile's first piece owns it; the following pieces are the first records of the
// next CTAs, up to the one that ends the tile.  blockIdx.y takes every fourth row.
constexpr int kKcThreads = 128;
template <int D, int ROWS>
__global__ void __launch_bounds__(kKcThreads)
kv4_combine_kernel(const AttnParams p, int ctas) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int s_count;
    const int c = blockIdx.x, tid = threadIdx.x;
    const int4 a = p.meta[2 * c], e = p.meta[2 * c + 1];
    int slot = -1;
    int4 me = a;
    if (a.x >= 0 && a.z == 0 && a.w > 0) slot = 2 * c;
    if (e.x >= 0 && e.z == 0 && e.w > 0) { slot = 2 * c + 1; me = e; }
    if (slot < 0) return;
    const Request r = kv4_request(p, me.x);
    const Units<ROWS> un = kv4_units<ROWS>(p, r);
    const int tile = me.y % un.tiles, kvh = me.y / un.tiles;
    if (tid == 0) s_count = ctas;
    __syncthreads();
    // the piece that ends the tile: the first of the following CTAs' first records with a negated end
    for (int j = c + 1 + tid; j < ctas; j += kKcThreads) {
        const int4 m = p.meta[2 * j];
        const bool end = m.x < 0 || m.w < 0 || m.y != me.y || m.x != me.x;
        if (end) atomicMin(&s_count, m.w < 0 && m.x == me.x && m.y == me.y ? j + 1 : j);
    }
    __syncthreads();
    const int last = s_count;                                     // pieces: slot, then 2j for c < j < last
    const int rows = min(ROWS, r.nq * p.group - tile * ROWS);
    const int n = ka_piece<D, ROWS>();
    constexpr int kPer = D / 4;                                   // threads per row: 4 channels each
    for (int x = tid; x < (ROWS / 4) * kPer; x += kKcThreads) {
        const int row = (x / kPer) * 4 + blockIdx.y, d0 = (x % kPer) * 4;
        if (row >= rows) continue;
        const float* first = p.part + static_cast<int64_t>(slot) * n;
        float mm = first[ROWS * D + row];
        for (int j = c + 1; j < last; ++j) mm = fmaxf(mm, p.part[static_cast<int64_t>(2 * j) * n + ROWS * D + row]);
        float ll = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int j = c; j < last; ++j) {
            const float* q = j == c ? first : p.part + static_cast<int64_t>(2 * j) * n;
            const float f = mm == -INFINITY ? 0.0f : ex2(q[ROWS * D + row] - mm);
            const float4 v = *reinterpret_cast<const float4*>(q + row * D + d0);
            ll += f * q[ROWS * D + ROWS + row];
            o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
        }
        const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
        const int64_t at = ka_out_row(p, r, kvh, tile * ROWS + row);
        *reinterpret_cast<uint2*>(p.out + at * D + d0) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (d0 == 0 && p.lse) p.lse[at] = ll > 0.0f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
    }
}

}  // namespace qat4
