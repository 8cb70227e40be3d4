// kv4_prefill.cuh -- the attention of kv4_attn.cuh for many query rows per
// request (prompts and chunks of prompts), on tcgen05 tensor cores.
//
// Bound: per (query row, key) pair and head 4 D flop on the tensor cores and one
// exponential; at D = 128 a 128 x 128 block is 1024 clocks of MMA at the dense
// bf16 rate and 1024 of the SM's 16 exponentials per clock, so both pipes have
// to run all the time.
//
// A work item is 256 query rows (token * group + head, as in the decode kernel)
// of one kv head, as two tiles of M = 128, over the keys that they see, in
// blocks of 128.  A CTA stays on its SM and takes item after item: the grid has
// one CTA per item, the last (longest) first, and a running CTA takes over the
// next one that has not started (clusterlaunchcontrol), so the end of one item
// overlaps the beginning of the next:
//   warps 0-3, 4-7  softmax of tile 0 / 1, one thread per row, 64 keys at a time:
//                   S from TMEM, the maximum, exp2, P back to TMEM as bf16 over its
//                   S (the A operand of the second product); O is rescaled in TMEM
//                   only when the maximum grows by more than 2^8
//   warps 8-11      decode the block's codes (one thread per token) into bf16
//                   operands in shared memory, double buffered
//   warps 12, 13    issue tile 0's / 1's MMAs: S = Q K^T (both K-major, N = 64) into
//                   two TMEM buffers, two steps ahead of the softmax, and
//                   O += P V (V as stored, MN-major)
//   warp 14         takes the next item
// The codes are decoded in the order (0, 4, 1, 5, 2, 6, 3, 7) of each 8
// channels, which needs no reordering of the packed words: Q is staged in the
// same order, and O's columns are put back in order on the way out.
//
// TMEM: S of tile x, buffer u in columns [128 x + 64 u, + 64), O of tile x in
// [256 + D x, + D).
//
// With few row tiles the keys of each are cut into `splits` equal parts, which
// leave (maximum, sum, unnormalised O) in the workspace for kv4_join_kernel.
// The keys of an item come in parts of kKpFold blocks, one after the other, which
// the CTA joins in the workspace itself.
//
// Measured on a B200 (calls replayed from a graph): a prompt of 4096 tokens with
// 32/8 heads of 128, 149 us = 924 TFLOP/s; three chunks of 1501 tokens on 4674 to
// 9001 cached ones with heads of 64, 377 us = 612 TFLOP/s.  What bounds it is the
// round trip of a step (scores, softmax, P, product, and the buffer's next
// scores), about 2000 clocks of which a thread's exponentials are 512: with them
// left out the two calls still take 133 and 334 us, with the MMAs cut to an
// eighth 104 and 267.  Tried and slower: one CTA per item without takeover (176
// and 457 us), scores of 128 keys in one buffer (174 and 525), two threads a row
// (161 and 512), weights taken against the maximum of the step before and redone
// when they overflow (158 and 473), separate warps for S and O (154 and 385),
// a quarter of the exponentials as polynomials (152 and 396).
#pragma once

#include "hessian.cuh"
#include "kv4_attn.cuh"

namespace qat4 {

constexpr int kKpThreads = 480;                    // 8 softmax, 4 decoding, 2 issuing warps, 1 for the items
constexpr int kKpRows = 256;
constexpr int kKpBlock = 128;                      // keys per block
constexpr uint32_t kKpHalf = 128 * 128;            // 128 rows x 64 channels bf16: 16 KB

template <int D>
struct KpLayout {
    static constexpr uint32_t kTile = (D / 64) * kKpHalf;          // 128 rows of D channels
    static constexpr uint32_t kQ = 0, kK = 2 * kTile, kV = 4 * kTile;
    static constexpr size_t kSmem = 6 * kTile + 1024;
    static constexpr uint32_t kO = 256;                            // TMEM columns
};

// Blocks of keys after which a work item is cut, the rows so far wait in the workspace, and O starts anew.  The tensor
// core cuts what it adds to the bits of the running sum: over n keys of like weights O comes out low by n 2^-27 of
// itself (measured: 7e-4 after 2^17 keys, 6.5e-3 after 2^20), by 2^-12 after the 2^15 keys here (1.5e-4).  The cut is
// between items, outside the steps' loop: folding O inside the loop took a prompt of 4096 tokens from 147 to 162 us.
constexpr int kKpFold = 256;

struct PrefillParams {
    AttnParams a;
    float* part;             // workspace: [splits][N * Hq][D], then maxima and sums [splits][N * Hq] each; null where
                             // splits is 1 and no request can have more than kKpFold blocks
    int splits;
};

// D[tmem] (+)= A[tmem] * B[smem], kind::f16, issued by a single thread.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
           "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
           "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// Row tiles of a request in this kernel.
__device__ __forceinline__ int kp_tiles(const AttnParams& p, const Request& r) {
    const int64_t rows = static_cast<int64_t>(r.nq) * p.group;
    return rows >= p.rows_lo && rows <= p.rows_hi ? static_cast<int>((rows + kKpRows - 1) / kKpRows) : 0;
}

// One token's codes and steps of keys or values.
template <int D>
struct KpRow {
    uint4 w[D / 32];
    uint32_t st[D / 64];
};
template <int D>
__device__ __forceinline__ void kp_load(KpRow<D>& r, const uint8_t* codes, const uint16_t* steps, int64_t cell, bool in) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) r.w[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) r.st[i] = 0u;
    if (in) {
        const uint4* c = reinterpret_cast<const uint4*>(codes + cell * (D / 2));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) r.w[i] = kv4_ld(c + i);
        const uint32_t* s = reinterpret_cast<const uint32_t*>(steps + cell * (D / 32));
#pragma unroll
        for (int i = 0; i < D / 64; ++i) r.st[i] = kv4_ld(s + i);
    }
}
// Groups FIRST .. LAST - 1 of a row decoded, each 8 channels in the order (0, 4, 1, 5, 2, 6, 3, 7).  The values are
// held in registers, so that the first half of a row is decoded before the wait for its buffer (a prompt of 4096
// tokens 147 us; 157 with all of it after the wait).
template <int D, int FIRST, int LAST>
struct KpValues {
    uint32_t x[16 * (LAST - FIRST)];
    __device__ __forceinline__ explicit KpValues(const KpRow<D>& r) {
#pragma unroll
        for (int i = FIRST; i < LAST; ++i) {
            const uint32_t st = __byte_perm(r.st[i >> 1], 0u, (i & 1) ? 0x3232 : 0x1010);
            const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t* const y = x + 16 * (i - FIRST) + 4 * j;
                y[0] = kv4_pair<0>(w[j], st);
                y[1] = kv4_pair<1>(w[j], st);
                y[2] = kv4_pair<2>(w[j], st);
                y[3] = kv4_pair<3>(w[j], st);
            }
        }
        // here, not where they are stored
#pragma unroll
        for (int i = 0; i < 16 * (LAST - FIRST); ++i) asm volatile("" : "+r"(x[i]));
    }
    // into operand row `row` (128-byte swizzle, 64 channels per 16 KB half)
    __device__ __forceinline__ void store(uint32_t base, int row) const {
        const uint32_t at = base + static_cast<uint32_t>(row) * 128u, s = static_cast<uint32_t>(row) & 7u;
#pragma unroll
        for (int c = 4 * FIRST; c < 4 * LAST; ++c) {
            const uint32_t* const y = x + 4 * (c - 4 * FIRST);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                         :: "r"(at + static_cast<uint32_t>(c >> 3) * kKpHalf + ((static_cast<uint32_t>(c & 7) ^ s) << 4)),
                            "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                         : "memory");
        }
    }
};

// A work item as its roles need it.
struct KpItem {
    int state;                // 1: work, -1: no more
    int b, kvh, row0, rows;   // request, kv head, first row and rows of the request
    int q0, len, first, lo;   // of the request (see Request)
    int t_first, n, split;    // first key, blocks of 128 keys
    int cut;                  // kKpRest: the rows' keys before these are in the workspace; kKpMore: others follow
};
enum : int { kKpRest = 1, kKpMore = 2 };

constexpr int kKpGroups = 2048;                    // 32 requests each
// Row tiles before each 32 requests, and all of them (`groups` + 1 entries), by a converged warp.
__device__ __noinline__ void kp_groups(const PrefillParams& pp, int* first, int groups, int lane) {
    int sum = 0;
    for (int g = 0; g < groups; ++g) {
        if (lane == 0) first[g] = sum;
        const int b = 32 * g + lane;
        sum += __reduce_add_sync(0xffffffffu, b < pp.a.B ? kp_tiles(pp.a, kv4_request(pp.a, b)) : 0);
    }
    if (lane == 0) first[groups] = sum;
    __syncwarp();
}
// Item `idx` of the grid, found by a converged warp: split, kv head, and the rank of its row tile, the
// last (longest) tile of a request first.  Requests are taken 32 by 32 (`first` has the tiles before each
// 32, when there are more), and of these from the longest to the shortest, so that short items even out the
// end.  False where there are fewer tiles.
__device__ __forceinline__ bool kp_locate(const PrefillParams& pp, const int* first, int groups, int idx, int lane, KpItem& it) {
    const AttnParams& p = pp.a;
    it.split = idx % pp.splits;
    const int hr = idx / pp.splits;
    it.kvh = hr % p.c.heads;
    int rank = hr / p.c.heads;
    int b0 = 0;
    if (groups > 1) {
        if (rank >= first[groups]) return false;
        int lo = 0, hi = groups;                                   // first[lo] <= rank < first[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= rank) lo = mid; else hi = mid;
        }
        b0 = 32 * lo;
        rank -= first[lo];
    }
    {
        const int b = b0 + lane;
        Request r = {0, 0, 0, 0, 0};
        if (b < p.B) r = kv4_request(p, b);
        const int n = b < p.B ? kp_tiles(p, r) : 0;
        int before = 0;                                            // tiles of the requests that come first
        for (int j = 0; j < 32 && b0 + j < p.B; ++j) {
            const int nj = __shfl_sync(0xffffffffu, n, j), lj = __shfl_sync(0xffffffffu, r.len, j);
            if (lj > r.len || (lj == r.len && j < lane)) before += nj;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, rank >= before && rank < before + n);
        if (hit == 0) return false;
        const int src = __ffs(hit) - 1;
        const int tile = n - 1 - (rank - before);                  // right in lane src
        it.state = 1;
        it.b = b0 + src;
        it.row0 = __shfl_sync(0xffffffffu, tile, src) * kKpRows;
        it.q0 = __shfl_sync(0xffffffffu, r.q0, src);
        it.rows = __shfl_sync(0xffffffffu, r.nq, src) * p.group;
        it.len = __shfl_sync(0xffffffffu, r.len, src);
        it.first = __shfl_sync(0xffffffffu, r.first, src);
        it.lo = __shfl_sync(0xffffffffu, r.lo, src);
        // keys that any row of the item sees, in blocks; this split's share of the blocks
        const int last_tok = (min(it.rows, it.row0 + kKpRows) - 1) / p.group, first_tok = it.row0 / p.group;
        const int hi = max(0, p.causal ? min(it.len, it.first + last_tok + 1) : it.len);
        const int lo = p.window > 0 ? max(0, it.first + first_tok - p.window + 1) : 0;
        const int blk0 = lo / kKpBlock, blocks = max(0, (hi + kKpBlock - 1) / kKpBlock - blk0);
        const int j0 = static_cast<int>(static_cast<int64_t>(blocks) * it.split / pp.splits);
        it.n = static_cast<int>(static_cast<int64_t>(blocks) * (it.split + 1) / pp.splits) - j0;
        it.t_first = (blk0 + j0) * kKpBlock;
        return true;
    }
}

template <int D>
__global__ void __launch_bounds__(kKpThreads, 1)
kv4_prefill_kernel(const PrefillParams pp) {
    using L = KpLayout<D>;
    const AttnParams& p = pp.a;
    extern __shared__ uint8_t kp_raw[];
    __shared__ __align__(16) uint4 clc_answer;
    __shared__ __align__(8) uint64_t k_full[2], v_full[2], k_free[2], v_free[2];
    __shared__ __align__(8) uint64_t s_full[2][2], p_full[2][2], o_full[2][2];     // [tile][buffer]
    __shared__ __align__(8) uint64_t q_full[2], item_full, item_free, clc_bar, done_bar[2];
    __shared__ KpItem s_item;
    __shared__ int s_first[kKpGroups + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(kp_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    pdl_launch_dependents();
    pdl_wait();
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 4);       // the decoding warps
            mbar_init(&v_full[i], 4);
            mbar_init(&k_free[i], 2);       // the issuing warps
            mbar_init(&v_free[i], 2);
            mbar_init(&q_full[i], 4);       // a tile's softmax warps
            mbar_init(&done_bar[i], 1);
            for (int u = 0; u < 2; ++u) {
                mbar_init(&s_full[i][u], 1);
                mbar_init(&p_full[i][u], 4);
                mbar_init(&o_full[i][u], 1);
            }
        }
        mbar_init(&item_full, 1);
        mbar_init(&item_free, 14);          // softmax, decoding and issuing warps
        mbar_init(&clc_bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    volatile int* abort = &abort_flag;
    const uint64_t limit = p.limit_ns;
    const int page = p.c.page, sh = __ffs(page) - 1;
    // waits of a converged warp: all lanes go on, or none
    auto wait = [&](uint64_t* bar, uint32_t phase) -> bool {
        return __all_sync(0xffffffffu, kv4_wait(bar, phase & 1u, abort, limit));
    };
    // The next item (k counts them); `release`: give the slot back at once.
    auto next_item = [&](KpItem& it, uint32_t k, bool release) -> bool {
        if (!wait(&item_full, k)) return false;
        it = s_item;
        __syncwarp();
        if (release && lane == 0) mbar_arrive(&item_free);
        return it.state > 0;
    };

    if (warp < 8) {
        // -------------------------------------------------------------- softmax
        const int x = warp >> 2;                           // tile
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const uint32_t ts = lanes + static_cast<uint32_t>(x) * 128u, to = lanes + L::kO + static_cast<uint32_t>(x) * D;
        const float c = p.scale_log2;
        const int64_t all = static_cast<int64_t>(p.N) * p.Hq;
        KpItem it;
        uint32_t cnt = 0;                                  // 64-key steps of this tile so far
        // the item before, whose rows are still in TMEM
        bool held = false, held_in = false;
        int held_n = 0, held_split = 0, held_cut = 0;
        int64_t held_at = 0;
        float m = -INFINITY, l = 0.0f;
        for (uint32_t k = 0;; ++k) {
            const bool more = next_item(it, k, true);
            const bool mine = more && (x == 0 || it.row0 + 128 < it.rows);
            const int row = it.row0 + x * 128 + (tid & 127);
            const bool in = mine && row < it.rows;
            const int tok = in ? row / p.group : 0;
            const int head = it.kvh * p.group + (in ? row - tok * p.group : 0);
            if (mine) {
                // this thread's row of Q, operand layout, channels in the decode's order.  The scores of the item
                // before have been waited for, so nothing reads the buffer any more.
                const uint4* src = reinterpret_cast<const uint4*>(p.q + (it.q0 + tok) * p.q_stride + static_cast<int64_t>(head) * D);
                const uint32_t at = sbase + L::kQ + x * L::kTile + static_cast<uint32_t>(tid & 127) * 128u;
                const uint32_t sw = static_cast<uint32_t>(tid) & 7u;
                uint4 v[D / 8];
#pragma unroll
                for (int w = 0; w < D / 8; ++w) {
                    v[w] = make_uint4(0u, 0u, 0u, 0u);
                    if (in) v[w] = kv4_ld(src + w);
                }
#pragma unroll
                for (int w = 0; w < D / 8; ++w)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                 :: "r"(at + static_cast<uint32_t>(w >> 3) * kKpHalf + ((static_cast<uint32_t>(w & 7) ^ sw) << 4)),
                                    "r"(__byte_perm(v[w].x, v[w].z, 0x5410)), "r"(__byte_perm(v[w].x, v[w].z, 0x7632)),
                                    "r"(__byte_perm(v[w].y, v[w].w, 0x5410)), "r"(__byte_perm(v[w].y, v[w].w, 0x7632))
                                 : "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[x]);
            }
            if (held) {
                // ---------------- the rows of the item before out, or their piece into the workspace
                if (held_n > 0) {
                    if (!wait(&o_full[x][(cnt - 1) & 1u], (cnt - 1) >> 1)) break;
                    tc_fence_after();
                }
                const bool whole = pp.splits == 1 && (held_cut & kKpMore) == 0;
                float* const piece = pp.part + (held_split * all + held_at) * D;
                float* const st = pp.part + pp.splits * all * D + held_split * all + held_at;
                float fo = 1.0f, fp = 0.0f;                // of O and of what is in the workspace
                if ((held_cut & kKpRest) && held_in) {
                    const float m0 = st[0], top = fmaxf(m, m0);
                    fo = top == -INFINITY ? 0.0f : ex2(m - top);
                    fp = top == -INFINITY ? 0.0f : ex2(m0 - top);
                    m = top;
                    l = fo * l + fp * st[pp.splits * all];
                }
                if (whole) {
                    const float f = l > 0.0f ? 1.0f / l : 0.0f;
                    fo *= f;
                    fp *= f;
                }
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    if (held_n > 0) {
                        tmem_ld_32x32b_x32(to + 32 * q, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0u;
                    }
                    if (!held_in) continue;
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)           // column 8w + (0..7) holds channel 8w + (0, 4, 1, 5, 2, 6, 3, 7)
                        v[(i & ~7) + ((i & 7) >> 1) + 4 * (i & 1)] = __uint_as_float(o[i]) * fo;
                    if (held_cut & kKpRest) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = fmaf(fp, piece[32 * q + i], v[i]);
                    }
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(p.out + held_at * D + 32 * q);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                                pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                    } else {
                        float4* dst = reinterpret_cast<float4*>(piece + 32 * q);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
                if (held_in) {
                    if (whole) {
                        if (p.lse) p.lse[held_at] = kv4_lse(m, l);
                    } else {
                        st[0] = m;
                        st[pp.splits * all] = l;
                    }
                }
                held = false;
            }
            if (!more) break;
            if (!mine) continue;
            const int pos = it.first + tok;
            // rows past the last query see everything: their zero queries are harmless, and masks stay rare
            const int lim = !in ? 0x7fffffff : p.causal ? pos : it.len - 1;
            const int low = in && p.window > 0 ? pos - p.window + 1 : 0;
            m = -INFINITY;
            l = 0.0f;
            const int steps = 2 * it.n;
            const int top = min(lim, it.len - 1);
            const int warp_top = __reduce_min_sync(0xffffffffu, top), warp_low = __reduce_max_sync(0xffffffffu, low);
            const int* const trow = p.table + it.b * p.table_stride;
            bool ok = true;
            // a lane's page of a block: -1 where the table names none (then its tokens are left out)
            auto entry = [&](int t0) -> int {
                const int t = t0 + lane * page;
                if (lane >= (kKpBlock >> sh) || t >= it.len) return 0;
                const int id = kv4_ld(trow + (t >> sh));
                return id < 0 || id >= p.c.pages ? -1 : 0;
            };
            int id = entry(it.t_first);
            uint32_t gone = 0;
            for (int i = 0; i < steps; ++i, ++cnt) {
                const int t0 = it.t_first + 64 * i;
                const uint32_t u = cnt & 1u, tsu = ts + 64u * u;
                if ((i & 1) == 0) {
                    gone = __ballot_sync(0xffffffffu, id < 0);
                    id = entry(t0 + kKpBlock);
                }
                ok = wait(&s_full[x][u], cnt >> 1);
                if (!ok) break;
                tc_fence_after();
                uint32_t s[64];
                tmem_ld_32x32b_x32(tsu, reinterpret_cast<uint32_t (&)[32]>(s[0]));
                tmem_ld_32x32b_x32(tsu + 32u, reinterpret_cast<uint32_t (&)[32]>(s[32]));
                tmem_ld_wait();
                if (gone != 0 || warp_top < t0 + 63 || warp_low > t0) {
                    const int in_block = 64 * (i & 1);
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        const int tk = t0 + e;
                        if (tk > top || tk < low || ((gone >> ((in_block + e) >> sh)) & 1u)) s[e] = 0xff800000u;   // -infinity
                    }
                }
                float mx[2] = {max3(s[0], s[1], s[2]), max3(s[3], s[4], s[5])};
#pragma unroll
                for (int e = 6; e < 62; e += 4) {
                    mx[0] = max3(__float_as_uint(mx[0]), s[e], s[e + 1]);
                    mx[1] = max3(__float_as_uint(mx[1]), s[e + 2], s[e + 3]);
                }
                const float xm = max3(__float_as_uint(fmaxf(mx[0], mx[1])), s[62], s[63]) * c;
                const bool grow = xm > m + kKaGrow;
                if (__any_sync(0xffffffffu, grow)) {
                    const float a = grow ? ex2(m - xm) : 1.0f;
                    if (grow) m = xm;
                    l *= a;
                    if (i > 0) {
                        // O holds the steps before: their products must have completed
                        ok = wait(&o_full[x][u ^ 1u], (cnt - 1) >> 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            uint32_t y[16];
                            tmem_ld_32x32b_x16(to + 16 * q, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * a);
                            tmem_st_32x32b_x16(to + 16 * q, y);
                        }
                    }
                }
                const float nm = m == -INFINITY ? 0.0f : -m;
                const float2 c2 = make_float2(c, c), n2 = make_float2(nm, nm);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                // P over its S (every lane of the warp has read its own)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 w = fma2(make_float2(__uint_as_float(s[32 * q + 2 * e]), __uint_as_float(s[32 * q + 2 * e + 1])), c2, n2);
                        w.x = ex2(w.x);
                        w.y = ex2(w.y);
                        sum[e & 1] = add2(sum[e & 1], w);
                        o[e] = pack_bf16(w.x, w.y);
                    }
                    tmem_st_32x32b_x16(tsu + 16u * q, o);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x][u]);
            }
            if (!ok) break;
            held = true;
            held_in = in;
            held_n = it.n;
            held_split = it.split;
            held_cut = it.cut;
            held_at = static_cast<int64_t>(it.q0 + tok) * p.Hq + head;
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------- decoding
        const int me = tid & 127;                          // token of the block
        constexpr int kHalf = D / 64;                      // groups in half a row
        KpItem it;
        uint32_t cnt = 0;                                  // blocks so far
        bool ok = true;
        for (uint32_t k = 0; ok && next_item(it, k, false); ++k) {
            auto cell_of = [&](int j, bool& live) -> int64_t {
                const int t = it.t_first + j * kKpBlock + me;
                live = j < it.n && t < it.len && t >= it.lo;
                int id = 0;
                if (live) {
                    id = kv4_ld(p.table + it.b * p.table_stride + (t >> sh));
                    live = id >= 0 && id < p.c.pages;
                }
                return (static_cast<int64_t>(id) * p.c.heads + it.kvh) * page + (t & (page - 1));
            };
            KpRow<D> kr, vr;
            bool live;
            int64_t cell = cell_of(0, live);
            kp_load<D>(kr, p.c.kc, p.c.ks, cell, live);
            kp_load<D>(vr, p.c.vc, p.c.vs, cell, live);
            const int last = max(0, it.n - 2);             // from here on the next item is wanted
            for (int j = 0; j < it.n; ++j, ++cnt) {
                if (j == last && lane == 0) mbar_arrive(&item_free);
                const uint32_t u = cnt & 1u, par = (cnt >> 1) ^ 1u;
                cell = cell_of(j + 1, live);
                const KpValues<D, 0, kHalf> k0(kr);
                ok = wait(&k_free[u], par);
                if (!ok) break;
                k0.store(sbase + L::kK + u * L::kTile, me);
                KpValues<D, kHalf, 2 * kHalf>(kr).store(sbase + L::kK + u * L::kTile, me);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&k_full[u]);
                kp_load<D>(kr, p.c.kc, p.c.ks, cell, live);
                const KpValues<D, 0, kHalf> v0(vr);
                ok = wait(&v_free[u], par);
                if (!ok) break;
                v0.store(sbase + L::kV + u * L::kTile, me);
                KpValues<D, kHalf, 2 * kHalf>(vr).store(sbase + L::kV + u * L::kTile, me);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_full[u]);
                kp_load<D>(vr, p.c.vc, p.c.vs, cell, live);
            }
            if (it.n == 0 && lane == 0) mbar_arrive(&item_free);
        }
    } else {
        if (warp < 14) {
            // ---------------------------------------------------------- products of tile x
            // The whole warp walks the loop and one elected lane issues, so addresses and descriptors stay
            // warp-uniform.  kind::f16, D float32, A and B bf16; S: N = 64, both K-major; O: N = D, B MN-major.
            constexpr uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
            constexpr uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((static_cast<uint32_t>(D) >> 3) << 17) |
                                      ((128u >> 4) << 24);
            const int x = warp - 12;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t dq = smem_desc_k_sw128(__shfl_sync(0xffffffffu, sbase, 0)) + ((L::kQ + x * L::kTile) >> 4);
            const uint64_t dk = smem_desc_k_sw128(__shfl_sync(0xffffffffu, sbase, 0)) + (L::kK >> 4);
            const uint64_t dv = smem_desc_mn_sw128(__shfl_sync(0xffffffffu, sbase, 0)) + (L::kV >> 4);
            const uint32_t ts = tm + x * 128u, to = tm + L::kO + x * D;
            const bool leader = elect_one();
            KpItem it;
            uint32_t cnt = 0, blk = 0, items = 0;          // this tile's 64-key steps, all blocks, this tile's items
            bool ok = true;
            for (uint32_t k = 0; ok && next_item(it, k, true); ++k) {
                if (x == 1 && it.row0 + 128 >= it.rows) {
                    // no rows in this tile: the blocks are the other tile's alone
                    for (int j = 0; ok && j < it.n; ++j, ++blk) {
                        ok = wait(&k_full[blk & 1u], blk >> 1) && wait(&v_full[blk & 1u], blk >> 1);
                        if (ok && leader) {
                            mbar_arrive(&k_free[blk & 1u]);
                            mbar_arrive(&v_free[blk & 1u]);
                        }
                        __syncwarp();
                    }
                    continue;
                }
                // scores of step i into buffer (cnt + i) & 1: keys 64 (i & 1) .. of block i / 2
                auto scores = [&](int i) -> bool {
                    const uint32_t bb = blk + static_cast<uint32_t>(i >> 1), u = (cnt + i) & 1u;
                    if ((i & 1) == 0 && !wait(&k_full[bb & 1u], bb >> 1)) return false;
                    tc_fence_after();
                    const uint64_t kb = dk + (((bb & 1u) * L::kTile + (i & 1) * 8192u) >> 4);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = (static_cast<uint32_t>(kk & 3) * 32u + static_cast<uint32_t>(kk >> 2) * kKpHalf) >> 4;
                            tc_mma_f16(ts + 64u * u, dq + off, kb + off, id_s, kk > 0);
                        }
                        tc_commit(&s_full[x][u]);
                        if (i & 1) tc_commit(&k_free[bb & 1u]);
                    }
                    __syncwarp();
                    return true;
                };
                const int steps = 2 * it.n;
                ok = wait(&q_full[x], items);
                ++items;
                for (int i = 0; ok && i < 2 && i < steps; ++i) {
                    // the item before: the product that reads this buffer's P
                    const uint32_t g = cnt + static_cast<uint32_t>(i);
                    ok = (g < 2 || wait(&o_full[x][g & 1u], (g - 2) >> 1)) && scores(i);
                }
                for (int i = 0; ok && i < steps; ++i) {
                    const uint32_t bb = blk + static_cast<uint32_t>(i >> 1), u = (cnt + i) & 1u;
                    if ((i & 1) == 0) ok = wait(&v_full[bb & 1u], bb >> 1);
                    ok = ok && wait(&p_full[x][u], (cnt + i) >> 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vb = dv + (((bb & 1u) * L::kTile + (i & 1) * 8192u) >> 4);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_f16_ts(to, ts + 64u * u + kk * 8, vb + (kk * 2048u >> 4), id_o, i > 0 || kk > 0);
                        tc_commit(&o_full[x][u]);
                        if (i & 1) tc_commit(&v_free[bb & 1u]);
                    }
                    __syncwarp();
                    if (i + 2 < steps) {
                        // the next scores of this buffer overwrite the P that the product above reads
                        ok = wait(&o_full[x][u], (cnt + i) >> 1) && scores(i + 2);
                    }
                }
                cnt += steps;
                blk += it.n;
            }
            // every MMA must have retired before TMEM is released
            if (leader) tc_commit(&done_bar[x]);
            __syncwarp();
            mbar_wait(&done_bar[x], 0, nullptr, kDrainLimitNs);
        } else if (warp == 14) {
            // ---------------------------------------------------------- the items
            const int groups = (p.B + 31) / 32;
            if (groups > 1) kp_groups(pp, s_first, groups, lane);
            int idx = static_cast<int>(blockIdx.x);
            uint32_t k = 0, asked = 0;
            bool ok = true, more = true;
            while (ok) {
                KpItem it;
                const bool work = more && kp_locate(pp, s_first, groups, idx, lane, it);
                if (work || !more) {
                    const int first = it.t_first, blocks = work ? it.n : 0;
                    for (int at = 0; at == 0 || at < blocks; at += kKpFold) {
                        if (k > 0) ok = wait(&item_free, k - 1);       // everyone has read the item before
                        if (!ok) break;
                        if (lane == 0) {
                            it.t_first = first + at * kKpBlock;
                            it.n = min(kKpFold, blocks - at);
                            it.cut = (at > 0 ? kKpRest : 0) | (at + kKpFold < blocks ? kKpMore : 0);
                            if (!more) it.state = -1;
                            s_item = it;
                            mbar_arrive(&item_full);
                        }
                        __syncwarp();
                        ++k;
                    }
                    if (!ok || !more) break;
                    ok = wait(&item_free, k - 1);                      // and wants the next one
                    if (!ok) break;
                }
                // take over the next CTA that has not started
                if (lane == 0) {
                    fence_proxy_async_smem();
                    mbar_arrive_expect_tx(&clc_bar, 16);
                    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                                 :: "r"(smem_u32(&clc_answer)), "r"(smem_u32(&clc_bar)) : "memory");
                }
                __syncwarp();
                ok = wait(&clc_bar, asked);
                if (!ok) break;
                ++asked;
                uint32_t got, cx;
                asm volatile(
                    "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t.reg .b32 y, z, w;\n\t"
                    "ld.shared.b128 a, [%2];\n\t"
                    "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
                    "selp.u32 %0, 1, 0, p;\n\t"
                    "mov.u32 %1, 0;\n\t"
                    "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, a;\n\t}"
                    : "=r"(got), "=r"(cx) : "r"(smem_u32(&clc_answer)) : "memory");
                __syncwarp();
                more = __shfl_sync(0xffffffffu, got, 0) != 0;
                idx = static_cast<int>(__shfl_sync(0xffffffffu, cx, 0));
            }
            // an answer may not land after the CTA is gone: every request has been waited for, or the limit has run out
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the splits of the rows that kv4_prefill_kernel computed: one warp per row and head.
constexpr int kKjThreads = 256;
template <int D>
__global__ void __launch_bounds__(kKjThreads)
kv4_join_kernel(const PrefillParams pp) {
    pdl_launch_dependents();
    pdl_wait();
    const AttnParams& p = pp.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t all = static_cast<int64_t>(p.N) * p.Hq;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * (kKjThreads / 32) + warp;
    if (at >= all) return;
    // rows of a request that another kernel computes, or of none, are not touched
    const int tok = static_cast<int>(at / p.Hq);
    bool mine = false;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        bool hit = false;
        if (b < p.B) {
            const Request r = kv4_request(p, b);
            hit = tok >= r.q0 && tok < r.q0 + r.nq && kp_tiles(p, r) > 0;
        }
        if (__any_sync(0xffffffffu, hit)) {
            mine = true;
            break;
        }
    }
    if (!mine) return;
    const float* st = pp.part + pp.splits * all * D;
    float mm = -INFINITY;
    for (int s = 0; s < pp.splits; ++s) mm = fmaxf(mm, st[s * all + at]);
    float ll = 0.0f, o[D / 32] = {};
    for (int s = 0; s < pp.splits; ++s) {
        const float f = mm == -INFINITY ? 0.0f : ex2(st[s * all + at] - mm);
        ll += f * st[(pp.splits + s) * all + at];
        const float* v = pp.part + (s * all + at) * D + lane * (D / 32);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] += f * v[i];
    }
    const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * D + lane * (D / 32));
#pragma unroll
    for (int i = 0; i < D / 32; i += 2) dst[i / 2] = pack_bf16(o[i] * inv, o[i + 1] * inv);
    if (lane == 0 && p.lse) p.lse[at] = kv4_lse(mm, ll);
}

}  // namespace qat4
