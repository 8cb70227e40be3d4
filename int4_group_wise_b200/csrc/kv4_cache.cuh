// kv4_cache.cuh -- the paged 4-bit key/value cache: its block tables and slot
// maps, the quantizing writer and the reader back.
//
// Format (decode on the INT4 grid of the model card "Opt.Gear-1B-qat-int4-per-
// channel-unquantized", section "Quantization Configuration": symmetric INT4,
// zero-point 0, here with one step per 32 channels of a token's head): codes
// uint8 [pages, heads, page, D/2] (channel 2j low nibble, 2j+1 high nibble, as
// the W4A16 export), steps bf16 [pages, heads, page, D/32].  A step that
// append writes has 5 significant bits, so code * step (3 + 5 bits) is exactly a
// bf16: the attention kernels feed the tensor cores with the cache's exact
// values.  Steps of other makers may have all 8 bits; their code * step is
// rounded to bf16 once.  The step is fl(m / 7) rounded UP to those 5 bits (m the group's largest
// magnitude), so no code is clipped; against an unrounded step the grid is up
// to 1/16 (on average 1/32) coarser.
#pragma once

#include <cuda_bf16.h>

#include "device_common.cuh"

namespace qat4 {

// A plain load.  These kernels may become resident before the kernel that writes what they read has run, so
// nothing of that goes through the read-only path, which supposes data that no one writes while the
// kernel lives: no read-only intrinsic, no restrict-qualified input.
template <typename T>
__device__ __forceinline__ T kv4_ld(const T* p) { return *p; }

// mbar_wait with its loop out of line: the kernels below wait in many places, and their code is kept small.
__device__ __noinline__ bool kv4_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    return mbar_wait(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool kv4_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    if (mbar_try_wait(smem_u32(bar), parity)) return true;
    return kv4_wait_slow(bar, parity, abort, limit_ns);
}

// The device's view of a cache.
struct Kv4View {
    uint8_t* kc;
    uint16_t* ks;
    uint8_t* vc;
    uint16_t* vs;
    int64_t pages;
    int page, heads, dim;
};

// ------------------------------------------------------------------ tables
// One step's bookkeeping, from request lengths alone:
//   have_b = ceil(len_b / P), need_b = ceil((len_b + new_b) / P), both at most
//   max_blocks; entry i in [have_b, need_b) of request b takes
//   free[sum_{b' < b} (need - have) + i - have_b], or -1 past the list's end;
//   cu = prefix sums of new; slot of token tok of request b = page * P + pos % P
//   with pos = len_b + tok - cu_b, or -1 where there is no page.
// Every CTA scans all B requests itself into shared memory (B is small against
// the tokens, and a second launch would cost more than the scan: 2-3 us), then
// takes its share of the table rows and of the tokens.  A new token's page is
// computed from the free list, not read from the table, so no CTA waits for
// another's writes.  Bound by latency: replayed from a graph, 32 requests
// with one token each take 6.0 us, of which the launch is about 1.5 and the scan (its
// divisions by the page size are 64-bit ones) most of the rest; 1000 requests with
// 511,000 tokens (2 MB written) 8.5.
constexpr int kTbThreads = 512;
constexpr int kTbMaxRequests = 16384;

struct TablesParams {
    const int* lengths;
    const int* fresh;        // new tokens per request
    int* table;
    int64_t table_stride;
    const int* free_pages;
    int* seq_lens;
    int* cu;
    int* slots;
    int* taken;
    int64_t num_slots;
    int B, max_blocks, num_free, page;
    int vec;                 // slots is 16-byte aligned: four tokens leave in one store
};

__host__ __device__ constexpr size_t tables_smem_bytes(int B) {
    return (2 * static_cast<size_t>(B) + 1) * 4;
}

__device__ __forceinline__ int tb_blocks(int64_t tokens, int page, int most) {
    const int64_t n = (tokens + page - 1) / page;
    return static_cast<int>(n < most ? n : most);
}

__global__ void __launch_bounds__(kTbThreads)
kv4_tables_kernel(const TablesParams p) {
    extern __shared__ int tb_smem[];
    int* const cu = tb_smem;              // [B + 1]
    int* const off = tb_smem + p.B + 1;   // [B] first free-list index of a request
    __shared__ int64_t wsum[2][kTbThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + kTbThreads - 1) / kTbThreads;
    const int r0 = min(p.B, tid * per), r1 = min(p.B, r0 + per);

    // sums of this thread's requests, then an exclusive scan over the block (64 bits: the totals of
    // wrong lengths may pass 2^31, and are cut there)
    int64_t n = 0, e = 0;
    for (int b = r0; b < r1; ++b) {
        const int len = max(0, p.lengths[b]), nw = max(0, p.fresh[b]);
        n += nw;
        e += tb_blocks(static_cast<int64_t>(len) + nw, p.page, p.max_blocks) - tb_blocks(len, p.page, p.max_blocks);
    }
    int64_t sn = n, se = e;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, sn, d), c = __shfl_up_sync(0xffffffffu, se, d);
        if (lane >= d) { sn += a; se += c; }
    }
    if (lane == 31) { wsum[0][warp] = sn; wsum[1][warp] = se; }
    __syncthreads();
    int64_t bn = sn - n, be = se - e, tn = 0, te = 0;
    for (int w = 0; w < kTbThreads / 32; ++w) {
        if (w < warp) { bn += wsum[0][w]; be += wsum[1][w]; }
        tn += wsum[0][w];
        te += wsum[1][w];
    }
    const int64_t top = 0x7fffffff;
    for (int b = r0; b < r1; ++b) {
        const int len = max(0, p.lengths[b]), nw = max(0, p.fresh[b]);
        cu[b] = static_cast<int>(bn < top ? bn : top);
        off[b] = static_cast<int>(be < top ? be : top);
        bn += nw;
        be += tb_blocks(static_cast<int64_t>(len) + nw, p.page, p.max_blocks) - tb_blocks(len, p.page, p.max_blocks);
    }
    if (tid == 0) cu[p.B] = static_cast<int>(tn < top ? tn : top);
    __syncthreads();

    // lengths, offsets and table rows: a warp per request
    if (blockIdx.x == 0) {
        for (int b = tid; b <= p.B; b += kTbThreads) p.cu[b] = cu[b];
        if (tid == 0) *p.taken = static_cast<int>(te < top ? te : top);
    }
    const int gwarp = blockIdx.x * (kTbThreads / 32) + warp, nwarps = gridDim.x * (kTbThreads / 32);
    for (int b = gwarp; b < p.B; b += nwarps) {
        const int len = max(0, p.lengths[b]);
        const int64_t total = static_cast<int64_t>(len) + max(0, p.fresh[b]);
        if (lane == 0) p.seq_lens[b] = static_cast<int>(total < top ? total : top);
        const int have = tb_blocks(len, p.page, p.max_blocks), need = tb_blocks(total, p.page, p.max_blocks);
        for (int i = have + lane; i < need; i += 32) {
            const int64_t f = static_cast<int64_t>(off[b]) + i - have;
            p.table[b * p.table_stride + i] = f < p.num_free ? p.free_pages[f] : -1;
        }
    }

    // slots, four consecutive tokens per thread; the request of the first by binary search
    const int sh = __ffs(p.page) - 1;
    const int64_t count = cu[p.B];
    for (int64_t t0 = 4 * (static_cast<int64_t>(blockIdx.x) * kTbThreads + tid); t0 < p.num_slots;
         t0 += 4 * static_cast<int64_t>(gridDim.x) * kTbThreads) {
        int out[4] = {-1, -1, -1, -1};
        if (t0 < count) {
            int lo = 0, hi = p.B;                      // cu[lo] <= t0 < cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t0) lo = mid; else hi = mid;
            }
            int b = lo;
            int len = max(0, p.lengths[b]), have = tb_blocks(len, p.page, p.max_blocks);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t tok = t0 + j;
                if (tok >= count) break;
                if (tok >= cu[b + 1]) {
                    do { ++b; } while (tok >= cu[b + 1]);
                    len = max(0, p.lengths[b]);
                    have = tb_blocks(len, p.page, p.max_blocks);
                }
                const int64_t pos = static_cast<int64_t>(len) + tok - cu[b];
                const int64_t blk = pos >> sh;
                if (blk >= p.max_blocks) continue;
                int64_t page = -1;
                if (blk < have) {
                    page = p.table[b * p.table_stride + blk];
                } else {
                    const int64_t f = off[b] + blk - have;
                    if (f < p.num_free) page = p.free_pages[f];
                }
                const int64_t slot = (page << sh) + (pos & (p.page - 1));
                if (page >= 0 && slot <= top) out[j] = static_cast<int>(slot);
            }
        }
        if (p.vec && t0 + 4 <= p.num_slots) {
            *reinterpret_cast<int4*>(p.slots + t0) = make_int4(out[0], out[1], out[2], out[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t0 + j < p.num_slots) p.slots[t0 + j] = out[j];
        }
    }
}

// ------------------------------------------------------------------ append
// Step of a group from its largest magnitude: fl(m / 7) with the 19 low of its
// 23 stored significand bits rounded up (the carry moves into the exponent), at
// most 2^100, and 0 below 2^-100 (then every code is 0).  The limits keep the
// step and its reciprocal away from overflow and subnormals.
__device__ __forceinline__ float kv4_step(float m) {
    const float d = __fdiv_rn(m, 7.0f);
    const float up = __uint_as_float((__float_as_uint(d) + 0x7FFFFu) & ~0x7FFFFu);
    return d < 0x1p-100f ? 0.0f : fminf(up, 0x1p100f);
}

// Eight values as packed codes, two's-complement nibbles, value i at bits 4i.  Any step and any values, which come
// in registers (an array by reference would be kept in local memory by the callers' common path too).
__device__ __forceinline__ uint32_t kv4_nibble(float v, float step) {
    return static_cast<uint32_t>(static_cast<int>(code_of(scaled_exact(v, step)))) & 15u;
}
__device__ __noinline__ uint32_t kv4_pack8_any(float4 a, float4 b, float step) {
    return kv4_nibble(a.x, step) | kv4_nibble(a.y, step) << 4 | kv4_nibble(a.z, step) << 8 | kv4_nibble(a.w, step) << 12 |
           kv4_nibble(b.x, step) << 16 | kv4_nibble(b.y, step) << 20 | kv4_nibble(b.z, step) << 24 | kv4_nibble(b.w, step) << 28;
}
// The same for groups without a NaN and with largest magnitude m at most 2^102, with the step.  There
// |v / step| < 7.001, so nothing is cut, and each code leaves as code + 8 in the low bits of
// 1.5 * 2^23 + 8 + code; multiplying the sum so far by 16 packs it in one integer FMA, and one subtraction
// and one exclusive or at the end take off what the words' upper bits and the eights have added.
// The quotients come from an approximate reciprocal r of the step (within 1 ulp):
// fl(m / 7), and float32 values, by Markstein's correction (P. Markstein, "Computation of elementary functions
//   on the IBM RISC System/6000 processor", 1990): q0 = fl(v r), e = v - q0 d exactly by one FMA, q = fl(q0 + e r).
//   A quotient of a 24-bit significand by one of at most 5 bits is at least 2^-31 of itself from the nearest
//   rounding boundary, and q0 + e r within 2^-44, so q is the IEEE quotient (below 2^-100, where e may lose bits,
//   the step is 0 and every code too).
// bf16 values need only which code is nearest.  v = V 2^a and step = S 2^b with V < 2^8, S < 2^5, so 2 v and
//   (2 k + 1) step, if they differ, differ by 2^(a + 1) or 2^b at least: v / step is k + 1/2 or farther than
//   2^-10 from it.  One FMA rounds v r to a multiple of 2^-11 (with 1.5 * 2^12 in front): exact halves become
//   exact halves again, the others stay on their side, and the addition of 1.5 * 2^23 rounds half to even.
__device__ __forceinline__ float kv4_quotient(float a, float d, float r) {
    const float q0 = __fmul_rn(a, r);
    return __fmaf_rn(__fmaf_rn(-q0, d, a), r, q0);
}
__device__ __forceinline__ float kv4_step_fast(float m, float& r) {
    const float d = kv4_quotient(m, 7.0f, 1.0f / 7.0f);
    const float up = __uint_as_float((__float_as_uint(d) + 0x7FFFFu) & ~0x7FFFFu);
    const float step = d < 0x1p-100f ? 0.0f : fminf(up, 0x1p100f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(step));
    if (step == 0.0f) r = 0.0f;                                       // then every quotient is 0
    return step;
}
template <bool BF16>
__device__ __forceinline__ uint32_t kv4_pack8(const float (&v)[8], float step, float r) {
    constexpr float kEight = 0x1.8p23f + 8.0f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        const float u = BF16 ? __fadd_rn(__fmaf_rn(v[i], r, 0x1.8p12f), kEight - 0x1.8p12f)
                             : __fadd_rn(kv4_quotient(v[i], step, r), kEight);
        w = w * 16u + __float_as_uint(u);
    }
    return (w - 0x4B400000u * 0x11111111u) ^ 0x88888888u;
}
// The larger one, NaN if either is.
__device__ __forceinline__ float kv4_max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint32_t kv4_max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Index of a token's item `at` of a head, where a token and head have `per` items (words of codes, steps).  One
// 64-bit product: the rest stays below 2^22 (1024 heads, pages of 128 tokens, 16 words).
__device__ __forceinline__ int64_t kv4_cell(const Kv4View& c, int sh, int slot, int head, uint32_t per, uint32_t at) {
    const uint32_t in = (static_cast<uint32_t>(head) << sh) + (slot & (c.page - 1));
    return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(slot >> sh)) * ((static_cast<uint32_t>(c.heads) << sh) * per) +
                                (in * per + at));
}

constexpr int kKvBlock = 256;
constexpr int kKvItems = 4;                        // gather: 8-channel words per thread of large batches, loaded together

// How blocks cover the words (or pairs of words) of n tokens of k (blockIdx.y = 0) or v (1): `tokens` whole tokens per block, or
// one token in `parts` blocks when it has more words than a block takes.
struct Kv4Span {
    uint32_t n;
    int row;                 // words of a token
    uint32_t inv;            // floor(2^32 / row) + 1: quotients of indexes below 2^16 by a multiply
    int tokens, parts, span; // span: words of a block
};
// Word `i` of this thread: its token, and the word inside the token; false past the end.
__device__ __forceinline__ bool kv4_word(const Kv4Span& s, int i, uint32_t& tok, int& rest) {
    const uint32_t li = threadIdx.x + kKvBlock * i;
    if (s.parts > 1) {
        tok = blockIdx.x / static_cast<uint32_t>(s.parts);
        rest = static_cast<int>(blockIdx.x - tok * s.parts) * s.span + static_cast<int>(li);
        return rest < s.row;
    }
    const uint32_t t = __umulhi(li, s.inv);
    rest = static_cast<int>(li - t * s.row);
    tok = blockIdx.x * static_cast<uint32_t>(s.tokens) + t;             // below 2^31 + 2^13
    return static_cast<int>(t) < s.tokens && tok < s.n;
}

// Thread = W words of 8 channels of a token and head, ITEMS times; 4 / W neighbouring lanes hold a group and find
// its largest magnitude by shuffles.  One pass: each value is read once, a thread's codes leave in one store.
// Bound: HBM, with the issue slots 70% busy.  16411 tokens of 8 heads of 128 (67 MB in, 19 MB out, 13.4 us at the
// copy rate), columns of a stacked projection, take 16.4 us with two times two words a thread (17.3 when the
// variants were measured: with 64-bit indexes throughout 17.9, one time two words 18.4, two times one 22.9, four
// times two 19.2).
template <bool BF16, int ITEMS, int W>
__global__ void __launch_bounds__(kKvBlock)
kv4_append_kernel(const Kv4View c, const Kv4Span s, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                  const int* slots) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kRaw = (BF16 ? 1 : 2) * W;                          // 16-byte loads per unit of W words
    const bool isv = blockIdx.y != 0;
    const char* const src = static_cast<const char*>(isv ? v : k);
    const uint32_t stride = static_cast<uint32_t>((isv ? v_stride : k_stride) / (BF16 ? 8 : 4));     // in 16 bytes
    const int lu = (c.dim == 128 ? 4 : 3) - (W == 2 ? 1 : 0), sh = __ffs(c.page) - 1;      // log2 of units per head
    uint4 raw[ITEMS][kRaw];
    int slot[ITEMS], at[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        uint32_t tok;
        slot[i] = -1;
#pragma unroll
        for (int h = 0; h < kRaw; ++h) raw[i][h] = make_uint4(0u, 0u, 0u, 0u);
        if (kv4_word(s, i, tok, at[i])) {
            // the values do not wait for the slot (rows without one are read for nothing)
            const uint4* a = reinterpret_cast<const uint4*>(src) + (static_cast<uint64_t>(tok) * stride + static_cast<uint32_t>(at[i] * kRaw));
#pragma unroll
            for (int h = 0; h < kRaw; ++h) raw[i][h] = __ldcs(a + h);
            slot[i] = kv4_ld(slots + tok);
            if ((slot[i] >> sh) >= c.pages) slot[i] = -1;
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        float x[W][8];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (BF16) {
                const uint32_t q[4] = {raw[i][w].x, raw[i][w].y, raw[i][w].z, raw[i][w].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[w][2 * j] = __uint_as_float(q[j] << 16);
                    x[w][2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
                }
            } else {
                const uint4 a = raw[i][(2 * w) % kRaw], b = raw[i][(2 * w + 1) % kRaw];
                x[w][0] = __uint_as_float(a.x); x[w][1] = __uint_as_float(a.y);
                x[w][2] = __uint_as_float(a.z); x[w][3] = __uint_as_float(a.w);
                x[w][4] = __uint_as_float(b.x); x[w][5] = __uint_as_float(b.y);
                x[w][6] = __uint_as_float(b.z); x[w][7] = __uint_as_float(b.w);
            }
        }
        // the group's largest magnitude, NaN if it holds one (bf16: magnitudes as integers, in pairs)
        float m = 0.0f;
        if (BF16) {
            uint32_t y = 0u;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                y = kv4_max_u16x2(y, kv4_max_u16x2(raw[i][w].x & 0x7FFF7FFFu, raw[i][w].y & 0x7FFF7FFFu));
                y = kv4_max_u16x2(y, kv4_max_u16x2(raw[i][w].z & 0x7FFF7FFFu, raw[i][w].w & 0x7FFF7FFFu));
            }
            m = kv4_max_nan(__uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u));
        } else {
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int j = 0; j < 8; ++j) m = kv4_max_nan(m, fabsf(x[w][j]));
        }
        m = kv4_max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));              // the 4 / W lanes of a group are in one
        if (W == 1) m = kv4_max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));  // token: it has a multiple of 8 words
        if (slot[i] < 0) continue;
        float step;
        uint32_t word[W];
        if (m <= 0x1p102f) {
            float r;
            step = kv4_step_fast(m, r);
#pragma unroll
            for (int w = 0; w < W; ++w) word[w] = kv4_pack8<BF16>(x[w], step, r);
        } else {
            // very large values, or a NaN, which does not count for the step; the group's lanes are all here
            constexpr int kLanes = 4 / W;
            const uint32_t lanes = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
            m = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[w][j]));
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, d));
            step = kv4_step(m);
#pragma unroll
            for (int w = 0; w < W; ++w)
                word[w] = kv4_pack8_any(make_float4(x[w][0], x[w][1], x[w][2], x[w][3]),
                                        make_float4(x[w][4], x[w][5], x[w][6], x[w][7]), step);
        }
        const int head = at[i] >> lu, u = at[i] & ((1 << lu) - 1);
        uint32_t* to = reinterpret_cast<uint32_t*>(isv ? c.vc : c.kc) + kv4_cell(c, sh, slot[i], head, W << lu, u * W);
        if (W == 2) *reinterpret_cast<uint2*>(to) = make_uint2(word[0], word[W - 1]);
        else *to = word[0];
        if ((u & (4 / W - 1)) == 0)
            (isv ? c.vs : c.ks)[kv4_cell(c, sh, slot[i], head, (W << lu) / 4, u / (4 / W))] = static_cast<uint16_t>(__float_as_uint(step) >> 16);
    }
}

// ------------------------------------------------------------------ gather
// Two bf16 values code * step from nibbles K and K + 4 of a word: a shift (none for K = 0), one logic op that
// flips the nibble's top bit and puts it into the significand of 16 (16 + (code + 8); K = 0: of 128), a packed
// subtraction that leaves the code exactly, and a packed product, rounded once, whatever the step.  Taking the
// offset off inside the product, fma(x, step, -24 step), saves the subtraction but is right for steps of at most 6
// significant bits only (3 step has to fit a bf16): it was 3% faster in the decode kernel (64 ragged requests 95 us
// for 97.6); looking at the steps first, to choose between the two, cost as much as the subtraction.
template <int K>
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, uint32_t step2) {
    const uint32_t v = K == 0 ? w : w >> (4 * K - 3);
    constexpr uint32_t kMask = K == 0 ? 0x000F000Fu : 0x00780078u, kZero = K == 0 ? 0x43084308u : 0x41C041C0u;
    uint32_t x, c, r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(x) : "r"(v), "r"(kMask), "r"(kZero));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(x), "r"(kZero));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(c), "r"(step2));
    return r;
}

// Thread = 8 channels of a token and head, ITEMS of them at a time: 4 bytes of codes in, 16 bytes out; rows
// without a slot are zero.  Bound: HBM (19 MB in and 67 MB out for 16411 tokens of 8 heads of 128: 13.4 us at the
// copy rate, 13.2 measured).
template <int ITEMS>
__global__ void __launch_bounds__(kKvBlock)
kv4_gather_kernel(const Kv4View c, const Kv4Span s, const int* slots, uint16_t* k, uint16_t* v) {
    pdl_launch_dependents();
    pdl_wait();
    const bool isv = blockIdx.y != 0;
    const int lw = c.dim == 128 ? 4 : 3, sh = __ffs(c.page) - 1;
    const uint32_t* const codes = reinterpret_cast<const uint32_t*>(isv ? c.vc : c.kc);
    const uint16_t* const steps = isv ? c.vs : c.ks;
    uint32_t q[ITEMS], st[ITEMS];
    int64_t to[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        uint32_t tok;
        int rest;
        to[i] = -1;
        q[i] = st[i] = 0;
        if (!kv4_word(s, i, tok, rest)) continue;
        to[i] = static_cast<int64_t>(static_cast<uint64_t>(tok) * static_cast<uint32_t>(s.row)) + rest;
        const int slot = kv4_ld(slots + tok);
        if (slot < 0 || (slot >> sh) >= c.pages) continue;
        const int head = rest >> lw, w = rest & ((1 << lw) - 1);
        q[i] = codes[kv4_cell(c, sh, slot, head, 1u << lw, w)];
        st[i] = steps[kv4_cell(c, sh, slot, head, 1u << (lw - 2), w >> 2)];
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        if (to[i] < 0) continue;
        const uint32_t s2 = st[i] | (st[i] << 16);
        const uint32_t a = kv4_pair<0>(q[i], s2), b = kv4_pair<1>(q[i], s2);      // channels (0, 4), (1, 5)
        const uint32_t e = kv4_pair<2>(q[i], s2), f = kv4_pair<3>(q[i], s2);      // (2, 6), (3, 7)
        __stcs(reinterpret_cast<uint4*>(isv ? v : k) + to[i],
               make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(e, f, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(e, f, 0x7632)));
    }
}

}  // namespace qat4
