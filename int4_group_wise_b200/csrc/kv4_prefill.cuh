// kv4_prefill.cuh -- the attention of kv4_attn.cuh for many query rows per
// request (prompts and chunks of prompts), on tcgen05 tensor cores.
//
// Bound: per (query row, key) pair and head 4 D flop on the tensor cores and one
// exponential; at D = 128 a 128 x 128 block is 1024 clocks of MMA at the dense
// bf16 rate and 1024 of the SM's 16 exponentials per clock, so both pipes have
// to run all the time.
//
// One CTA (one per SM) owns 256 query rows (token * group + head, as in the
// decode kernel) of one kv head as two tiles of M = 128, and walks its keys in
// blocks of 128:
//   warps 0-3, 4-7  softmax of tile 0 / 1, one thread per row: S from TMEM, row
//                   maximum, exp2, P back to TMEM as bf16 (the A operand of the
//                   second product), O rescaled in TMEM only when the maximum
//                   grows by more than 2^8
//   warps 8-11      decode the block's codes (one thread per token) into bf16
//                   operands in shared memory, double buffered
//   warp 12         issues the MMAs: S = Q K^T (both K-major) and O += P V (V as
//                   stored, MN-major); tile 0's products run while tile 1's
//                   softmax does, and the other way round
// The codes are decoded in the order (0, 4, 1, 5, 2, 6, 3, 7) of each 8
// channels, which needs no reordering of the packed words: Q is staged in the
// same order, and O's columns are put back in order on the way out.
//
// TMEM: S of both tiles [0, 256), O [256, 256 + 2 D); P overlays its S at
// D = 128 (the next S of a tile is issued after the product that reads P, in
// order and of the same shape) and has columns of its own at D = 64.
//
// With few row tiles the keys of each are cut into `splits` equal parts (grid
// y), which leave (maximum, sum, unnormalised O) in the workspace for
// kv4_join_kernel.
#pragma once

#include "hessian.cuh"
#include "kv4_attn.cuh"

namespace qat4 {

constexpr int kKpThreads = 512;                    // 2 softmax warpgroups, 1 decoding, 1 issuing
constexpr int kKpRegsSoftmax = 184, kKpRegsDecode = 96, kKpRegsIssue = 40;   // per thread; their sum over the four
                                                   // warpgroups is below the 128 per thread of the launch
constexpr int kKpRows = 256;
constexpr int kKpBlock = 128;                      // keys per block
constexpr uint32_t kKpHalf = 128 * 128;            // 128 rows x 64 channels bf16: 16 KB

template <int D>
struct KpLayout {
    static constexpr uint32_t kTile = (D / 64) * kKpHalf;          // 128 rows of D channels
    static constexpr uint32_t kQ = 0, kK = 2 * kTile, kV = 4 * kTile;
    static constexpr size_t kSmem = 6 * kTile + 1024;
    static constexpr uint32_t kO = 256;                            // TMEM columns
    static constexpr uint32_t kP = D == 128 ? 0 : 256 + 2 * D;
    static constexpr uint32_t kPStride = D == 128 ? 128 : 64;
};

struct PrefillParams {
    AttnParams a;
    float* part;             // workspace: [splits][N * Hq][D], then maxima and sums [splits][N * Hq] each
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

// Row tiles of a request in this kernel.
__device__ __forceinline__ int kp_tiles(const AttnParams& p, const Request& r) {
    const int64_t rows = static_cast<int64_t>(r.nq) * p.group;
    return rows >= p.rows_lo && rows <= p.rows_hi ? static_cast<int>((rows + kKpRows - 1) / kKpRows) : 0;
}

// Eight codes as 16 bytes of bf16 in the order (0, 4, 1, 5, 2, 6, 3, 7).
__device__ __forceinline__ void kp_store8(uint32_t addr, uint32_t w, uint32_t s2, uint32_t o2) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 :: "r"(addr), "r"(kv4_pair(w << 3, s2, o2)), "r"(kv4_pair(w >> 1, s2, o2)),
                    "r"(kv4_pair(w >> 5, s2, o2)), "r"(kv4_pair(w >> 9, s2, o2))
                 : "memory");
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
        for (int i = 0; i < D / 32; ++i) r.w[i] = __ldg(c + i);
        const uint32_t* s = reinterpret_cast<const uint32_t*>(steps + cell * (D / 32));
#pragma unroll
        for (int i = 0; i < D / 64; ++i) r.st[i] = __ldg(s + i);
    }
}
// The row as operand row `row` (128-byte swizzle, 64 channels per 16 KB half).
template <int D>
__device__ __forceinline__ void kp_decode(const KpRow<D>& r, uint32_t base, int row) {
    const uint32_t at = base + static_cast<uint32_t>(row) * 128u, x = static_cast<uint32_t>(row) & 7u;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint32_t st = __byte_perm(r.st[i >> 1], 0u, (i & 1) ? 0x3232 : 0x1010), o2 = kv4_off(st);
        const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t c = static_cast<uint32_t>(4 * i + j);       // 8-channel word of the row
            kp_store8(at + (c >> 3) * kKpHalf + (((c & 7u) ^ x) << 4), w[j], st, o2);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kKpThreads, 1)
kv4_prefill_kernel(const PrefillParams pp) {
    using L = KpLayout<D>;
    const AttnParams& p = pp.a;
    extern __shared__ uint8_t kp_raw[];
    __shared__ __align__(8) uint64_t k_full[2], v_full[2], k_free[2], v_free[2], s_full[2], p_full[2], o_full[2];
    __shared__ __align__(8) uint64_t q_full, done_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, s_b, s_tile;
    __shared__ int scan[kKpThreads / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(kp_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    pdl_launch_dependents();
    pdl_wait();

    // ---- this CTA's row tile: the last ones first (they see the most keys)
    const int per = (p.B + kKpThreads - 1) / kKpThreads;
    const int rb0 = min(p.B, tid * per), rb1 = min(p.B, rb0 + per);
    int mine = 0;
    for (int b = rb0; b < rb1; ++b) mine += kp_tiles(p, kv4_request(p, b));
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += a;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 4);       // the decoding warps
            mbar_init(&v_full[i], 4);
            mbar_init(&k_free[i], 1);
            mbar_init(&v_free[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);       // a tile's softmax warps
            mbar_init(&o_full[i], 1);
        }
        mbar_init(&q_full, 8);
        mbar_init(&done_bar, 1);
        abort_flag = 0;
        s_b = -1;
        fence_mbar_init();
    }
    __syncthreads();
    int before = incl - mine, total = 0;
    for (int w = 0; w < kKpThreads / 32; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    const int kvh = static_cast<int>(blockIdx.x) % p.c.heads;
    const int want = total - 1 - static_cast<int>(blockIdx.x) / p.c.heads;
    if (want >= before && want < before + mine) {
        int at = before;
        for (int b = rb0; b < rb1; ++b) {
            const int n = kp_tiles(p, kv4_request(p, b));
            if (want < at + n) {
                s_b = b;
                s_tile = want - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    if (s_b < 0) return;
    const int b = s_b;
    const Request r = kv4_request(p, b);
    const int rows = r.nq * p.group, row0 = s_tile * kKpRows;
    const bool two = row0 + 128 < rows;                    // the second tile has rows
    // keys that any row of the CTA sees, in blocks; this split's share of the blocks
    const int last_tok = (min(rows, row0 + kKpRows) - 1) / p.group, first_tok = row0 / p.group;
    const int hi = max(0, p.causal ? min(r.len, r.first + last_tok + 1) : r.len);
    const int lo = p.window > 0 ? max(0, r.first + first_tok - p.window + 1) : 0;
    const int blk0 = lo / kKpBlock, blocks = max(0, (hi + kKpBlock - 1) / kKpBlock - blk0);
    const int split = blockIdx.y;
    const int j0 = static_cast<int>(static_cast<int64_t>(blocks) * split / pp.splits);
    const int n = static_cast<int>(static_cast<int64_t>(blocks) * (split + 1) / pp.splits) - j0;
    const int t_first = (blk0 + j0) * kKpBlock;
    const int page = p.c.page, sh = __ffs(page) - 1;

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

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kKpRegsSoftmax));
        // -------------------------------------------------------------- softmax
        const int x = warp >> 2;                           // tile
        const int row = row0 + x * 128 + (tid & 127);
        const bool in = row < rows;
        const int tok = in ? row / p.group : 0;
        const int head = kvh * p.group + (in ? row - tok * p.group : 0);
        {
            // this thread's row of Q, operand layout, channels in the decode's order
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (r.q0 + tok) * p.q_stride + static_cast<int64_t>(head) * D);
            const uint32_t at = sbase + L::kQ + x * L::kTile + static_cast<uint32_t>(tid & 127) * 128u;
            const uint32_t sw = static_cast<uint32_t>(tid) & 7u;
#pragma unroll
            for (int w = 0; w < D / 8; ++w) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (in) v = __ldg(src + w);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                             :: "r"(at + static_cast<uint32_t>(w >> 3) * kKpHalf + ((static_cast<uint32_t>(w & 7) ^ sw) << 4)),
                                "r"(__byte_perm(v.x, v.z, 0x5410)), "r"(__byte_perm(v.x, v.z, 0x7632)),
                                "r"(__byte_perm(v.y, v.w, 0x5410)), "r"(__byte_perm(v.y, v.w, 0x7632))
                             : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);
        }
        const int pos = r.first + tok;
        // rows past the last query see everything: their zero queries are harmless, and masks stay rare
        const int lim = !in ? 0x7fffffff : p.causal ? pos : r.len - 1;
        const int low = in && p.window > 0 ? pos - p.window + 1 : 0;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const uint32_t ts = lanes + static_cast<uint32_t>(x) * 128u, to = lanes + L::kO + static_cast<uint32_t>(x) * D;
        const uint32_t tp = lanes + L::kP + static_cast<uint32_t>(x) * L::kPStride;
        const float c = p.scale_log2;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        const int np = kKpBlock >> sh;                     // pages per block
        for (int j = 0; j < n && (x == 0 || two); ++j) {
            const int t0 = t_first + j * kKpBlock;
            // pages the table does not name (checked by the first lanes while the scores are computed)
            int id = 0;
            if (lane < np && t0 + lane * page < r.len) {
                id = __ldg(p.table + b * p.table_stride + ((t0 >> sh) + lane));
                id = id < 0 || id >= p.c.pages ? -1 : 0;
            }
            const uint32_t gone = __ballot_sync(0xffffffffu, id < 0);
            ok = mbar_wait(&s_full[x], static_cast<uint32_t>(j) & 1u, abort, limit);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(ts + 32 * q, s[q]);
            tmem_ld_wait();
            const bool plain = gone == 0 && t0 + kKpBlock <= r.len && lim >= t0 + kKpBlock - 1 && low <= t0;
            if (!__all_sync(0xffffffffu, plain)) {
                const int top = min(lim, r.len - 1);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int tk = t0 + 32 * q + i;
                        if (tk > top || tk < low || ((gone >> ((32 * q + i) >> sh)) & 1u)) s[q][i] = 0xff800000u;   // -inf
                    }
            }
            float mx[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                mx[q] = fmaxf(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]));
#pragma unroll
                for (int i = 2; i < 32; i += 2)
                    mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])));
            }
            const float xm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            const bool grow = xm > m + kKaGrow;
            if (__any_sync(0xffffffffu, grow)) {
                const float a = grow ? ex2(m - xm) : 1.0f;
                if (grow) m = xm;
                l *= a;
                if (j > 0) {
                    // the product of the block before has completed: it was issued before this block's scores
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(to + 32 * q, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                        tmem_st_32x32b_x32(to + 32 * q, o);
                    }
                }
            }
            const float nm = m == -INFINITY ? 0.0f : -m;
            const float2 c2 = make_float2(c, c), n2 = make_float2(nm, nm);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float2 e = fma2(make_float2(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1])), c2, n2);
                    e.x = ex2(e.x);
                    e.y = ex2(e.y);
                    sum[i & 1] = add2(sum[i & 1], e);
                    o[i] = pack_bf16(e.x, e.y);
                }
                tmem_st_32x32b_x16(tp + 16 * q, o);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[x]);
        }
        // ---------------- the rows out, or their piece into the workspace
        if (x == 0 || two) {
            if (n > 0 && ok) {
                ok = mbar_wait(&o_full[x], 0, abort, limit);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
            }
            const int64_t at = static_cast<int64_t>(r.q0 + tok) * p.Hq + head;
            const int64_t all = static_cast<int64_t>(p.N) * p.Hq;
            const bool whole = pp.splits == 1;
            const float f = !whole ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
            if (ok) {
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld_32x32b_x32(to + 32 * q, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0u;
                    }
                    if (!in) continue;
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)           // column 8w + (0..7) holds channel 8w + (0, 4, 1, 5, 2, 6, 3, 7)
                        v[(i & ~7) + ((i & 7) >> 1) + 4 * (i & 1)] = __uint_as_float(o[i]) * f;
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + 32 * q);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                                pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                    } else {
                        float4* dst = reinterpret_cast<float4*>(pp.part + (split * all + at) * D + 32 * q);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
                if (in) {
                    if (whole) {
                        if (p.lse) p.lse[at] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
                    } else {
                        float* st = pp.part + pp.splits * all * D;
                        st[split * all + at] = m;
                        st[(pp.splits + split) * all + at] = l;
                    }
                }
            }
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kKpRegsDecode));
        // ------------------------------------------------------------- decoding
        const int me = tid & 127;                          // token of the block
        auto cell_of = [&](int j, bool& live) -> int64_t {
            const int t = t_first + j * kKpBlock + me;
            live = j < n && t < r.len && t >= r.lo;
            int id = 0;
            if (live) {
                id = __ldg(p.table + b * p.table_stride + (t >> sh));
                live = id >= 0 && id < p.c.pages;
            }
            return (static_cast<int64_t>(id) * p.c.heads + kvh) * page + (t & (page - 1));
        };
        KpRow<D> kr, vr;
        bool live;
        int64_t cell = cell_of(0, live);
        kp_load<D>(kr, p.c.kc, p.c.ks, cell, live);
        kp_load<D>(vr, p.c.vc, p.c.vs, cell, live);
        for (int j = 0; j < n; ++j) {
            const int u = j & 1;
            const uint32_t par = (static_cast<uint32_t>(j >> 1) & 1u) ^ 1u;
            cell = cell_of(j + 1, live);
            bool ok = mbar_wait(&k_free[u], par, abort, limit);
            if (!__all_sync(0xffffffffu, ok)) break;
            kp_decode<D>(kr, sbase + L::kK + u * L::kTile, me);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_full[u]);
            kp_load<D>(kr, p.c.kc, p.c.ks, cell, live);
            ok = mbar_wait(&v_free[u], par, abort, limit);
            if (!__all_sync(0xffffffffu, ok)) break;
            kp_decode<D>(vr, sbase + L::kV + u * L::kTile, me);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_full[u]);
            kp_load<D>(vr, p.c.vc, p.c.vs, cell, live);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kKpRegsIssue));
        if (warp == 12 && lane == 0) {
            // ---------------------------------------------------------- products
            // kind::f16, D float32, A and B bf16; S: N = 128, both K-major; O: N = D, B MN-major
            constexpr uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
            constexpr uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((static_cast<uint32_t>(D) >> 3) << 17) |
                                      ((128u >> 4) << 24);
            auto scores = [&](int x, int j) {
                const uint32_t qa = sbase + L::kQ + x * L::kTile, kb = sbase + L::kK + (j & 1) * L::kTile;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = static_cast<uint32_t>(kk & 3) * 32u + static_cast<uint32_t>(kk >> 2) * kKpHalf;
                    tc_mma_f16(tmem + x * 128u, smem_desc_k_sw128(qa + off), smem_desc_k_sw128(kb + off), id_s, kk > 0);
                }
                tc_commit(&s_full[x]);
            };
            auto output = [&](int x, int j) {
                const uint32_t vb = sbase + L::kV + (j & 1) * L::kTile;
#pragma unroll
                for (int kk = 0; kk < kKpBlock / 16; ++kk)
                    tc_mma_f16_ts(tmem + L::kO + x * D, tmem + L::kP + x * L::kPStride + kk * 8,
                                  smem_desc_mn_sw128(vb + kk * 2048u), id_o, j > 0 || kk > 0);
            };
            const int tiles = two ? 2 : 1;
            bool ok = n > 0 && mbar_wait(&q_full, 0, abort, limit) && mbar_wait(&k_full[0], 0, abort, limit);
            if (ok) {
                tc_fence_after();
                for (int x = 0; x < tiles; ++x) scores(x, 0);
                tc_commit(&k_free[0]);
            }
            for (int j = 0; ok && j < n; ++j) {
                const uint32_t par = static_cast<uint32_t>(j >> 1) & 1u;
                ok = mbar_wait(&v_full[j & 1], par, abort, limit);
                for (int x = 0; ok && x < tiles; ++x) {
                    ok = mbar_wait(&p_full[x], static_cast<uint32_t>(j) & 1u, abort, limit);
                    if (!ok) break;
                    tc_fence_after();
                    output(x, j);
                    if (x == tiles - 1) tc_commit(&v_free[j & 1]);
                    if (j + 1 == n) {
                        tc_commit(&o_full[x]);
                        continue;
                    }
                    if (x == 0) {
                        ok = mbar_wait(&k_full[(j + 1) & 1], static_cast<uint32_t>((j + 1) >> 1) & 1u, abort, limit);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    scores(x, j + 1);
                    if (x == tiles - 1) tc_commit(&k_free[(j + 1) & 1]);
                }
            }
            // every MMA must have retired before TMEM is released
            tc_commit(&done_bar);
            mbar_wait(&done_bar, 0, nullptr, kDrainLimitNs);
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
    if (lane == 0 && p.lse) p.lse[at] = ll > 0.0f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace qat4
