// tfa_rope.cu -- norms of queries and keys for each head with the rotary
// position in the same pass, and its gradient.
//
// For a head row x of D channels at position p (all in fp32, rounded to bf16
// once at the end):
//   y = x r w,  r = 1 / sqrt(mean(x^2) + eps)         (y = x without weights)
//   (o_a, o_b) = m (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = p f_i
// for the rot / 2 pairs i: channels (i, i + rot / 2), or (2i, 2i + 1) where the
// pairs are interleaved; channels from rot on pass through.
// The angle is taken in 64 bits, reduced to a fraction of a turn there and only
// then rounded: p f_i in fp32 would be off by p f_i 2^-24 radians, 0.06 at
// position 10^6.
// Gradient, with g the rotated-back dy (the transposed rotation) and h = x r:
//   dw += g h,   dx = r (w g - h mean(w g h)).
//
// Layout: a row is D / 8 lanes of two times 8 bytes, so a warp instruction moves whole
// 128-byte lines; tokens come in the projection's order ([B, L, H, D], any
// strides) and leave in the attention's ([B, H, L, D], or a cache's rows), so
// no separate transpose reads the data again.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/tfa.h"
#include "tfa_internal.h"
#include "tfa_ptx.cuh"

namespace tfa {
namespace rope {

constexpr int kThreads = 256;
constexpr int kBwdBlocks = 296;  // gradient kernel: most blocks, so most partial sums of a weight

struct Strides {
    long long b, l, h;  // elements
};
struct Params {
    const __nv_bfloat16 *q, *k;    // forward: inputs; gradient: the forward's inputs
    const __nv_bfloat16 *dq, *dk;  // gradient: upstream
    __nv_bfloat16 *qo, *ko;
    Strides sq, sk, sdq, sdk, sqo, sko;
    const __nv_bfloat16 *wq, *wk;
    const double *inv_freq;
    const int *pos;
    int pos_per_row, pos0;
    int B, L, Hq, Hkv, rot;
    int rows_per_block;  // forward: head rows of a token that one block takes
    float eps, mscale;
    int conj;   // rotate back (a gradient)
    int inter;  // pairs of neighbouring channels (2i, 2i + 1)
    float *partial;  // gradient: [blocks][D]
    int q_blocks;    // gradient: blocks that take query rows, the first ones
};

// 64 bits: a row behind a first position near 2^31 lies past an int.
__device__ __forceinline__ long long position(const Params &p, int b, int l) {
    if (!p.pos) return static_cast<long long>(p.pos0) + l;
    return p.pos_per_row ? load_input<true>(p.pos + static_cast<long long>(b) * p.L + l)
                         : static_cast<long long>(load_input<true>(p.pos + b)) + l;
}

// The cosines and sines of a position's pairs, times mscale; a gradient's sines are negated.
template <int D>
struct Table {
    float c[D / 2], s[D / 2];
};
__device__ __forceinline__ double turns_per_token(const Params &p, int i) {
    constexpr double kInv2Pi = 0.15915494309189533577;
    return p.inv_freq[i] * kInv2Pi;
}
template <int D>
__device__ __forceinline__ void angle(const Params &p, long long pos, double per_token, int i, Table<D> &tab) {
    double turns = static_cast<double>(pos) * per_token;
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * static_cast<float>(turns), &s, &c);
    tab.c[i] = c * p.mscale;
    tab.s[i] = s * (p.conj ? -p.mscale : p.mscale);
}

// Lane `lane` of a row holds channels a .. a+3 and b .. b+3, chosen so that it holds
// both channels of its pairs 4 lane .. 4 lane + 3: no lane needs another's values.
struct Channels {
    int a, b;
    bool turns;  // a pair's channels; else they pass through
    __device__ __forceinline__ Channels(const Params &p, int lane) {
        turns = lane * 8 < p.rot;
        a = turns && !p.inter ? lane * 4 : lane * 8;
        b = turns && !p.inter ? a + (p.rot >> 1) : a + 4;
    }
};

// Eight channels as fp32 pairs: channels a, a+1 | a+2, a+3 | b, b+1 | b+2, b+3.
struct Eight {
    float2 v[4];
};
__device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ Eight unpack(uint2 a, uint2 b) {
    return Eight{{unpack(a.x), unpack(a.y), unpack(b.x), unpack(b.y)}};
}
__device__ __forceinline__ uint32_t pack(float2 v) { return pack_bf16(v.x, v.y); }
__device__ __forceinline__ Eight load_eight(const __nv_bfloat16 *row, const Channels &ch) {
    return unpack(*reinterpret_cast<const uint2 *>(row + ch.a), *reinterpret_cast<const uint2 *>(row + ch.b));
}
__device__ __forceinline__ void store_eight(__nv_bfloat16 *row, const Channels &ch, const Eight &x) {
    *reinterpret_cast<uint2 *>(row + ch.a) = make_uint2(pack(x.v[0]), pack(x.v[1]));
    *reinterpret_cast<uint2 *>(row + ch.b) = make_uint2(pack(x.v[2]), pack(x.v[3]));
}

// The lane's four pairs' factors.
template <int D, bool INTER>
struct Factors {
    float4 c, s;
    __device__ __forceinline__ void load(const Table<D> &tab, int lane) {
        c = *reinterpret_cast<const float4 *>(tab.c + lane * 4);
        s = *reinterpret_cast<const float4 *>(tab.s + lane * 4);
    }
    __device__ __forceinline__ void rotate(Eight &x) const {
        const float2 c2[2] = {{c.x, c.y}, {c.z, c.w}}, s2[2] = {{s.x, s.y}, {s.z, s.w}};
        if constexpr (INTER) {
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 y = x.v[e];
                x.v[e] = make_float2(fmaf(y.x, cc[e], -y.y * ss[e]), fmaf(y.y, cc[e], y.x * ss[e]));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 a = x.v[e], b = x.v[2 + e];
                x.v[e] = fma2(a, c2[e], mul2(b, make_float2(-s2[e].x, -s2[e].y)));
                x.v[2 + e] = fma2(b, c2[e], mul2(a, s2[e]));
            }
        }
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Both sums at once: a half of the row's lanes goes on with each, until the last exchange.
template <int LPR>
__device__ __forceinline__ void row_sums(float &x, float &y) {
    const bool upper = threadIdx.x & (LPR / 2);
    float mine = upper ? y : x;
    mine += __shfl_xor_sync(0xffffffffu, upper ? x : y, LPR / 2);
#pragma unroll
    for (int o = LPR / 4; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    const float other = __shfl_xor_sync(0xffffffffu, mine, LPR / 2);
    x = upper ? other : mine;
    y = upper ? mine : other;
}

template <int D, bool NORM, bool INTER>
__global__ void __launch_bounds__(kThreads, 5) forward_kernel(const __grid_constant__ Params p) {
    constexpr int LPR = D / 8, kSlots = kThreads / LPR;
    __shared__ __align__(16) Table<D> tab;
    const int token = blockIdx.x, b = token / p.L, l = token - b * p.L;
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const Channels ch(p, lane);
    const int n_rows = p.Hq + p.Hkv;
    const int row0 = blockIdx.y * p.rows_per_block;
    const int row1 = min(row0 + p.rows_per_block, n_rows);
    const __nv_bfloat16 *q = p.q + b * p.sq.b + l * p.sq.l;
    const __nv_bfloat16 *k = p.k + b * p.sk.b + l * p.sk.l;
    __nv_bfloat16 *qo = p.qo + b * p.sqo.b + l * p.sqo.l;
    __nv_bfloat16 *ko = p.ko + b * p.sko.b + l * p.sko.l;
    grid_dep_wait();
    grid_dep_launch();
    // the first rows are on their way while the table is computed
    constexpr int kAhead = 2;
    uint2 xa[kAhead], xb[kAhead];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int row = base + slot + u * kSlots;
            xa[u] = xb[u] = make_uint2(0u, 0u);
            if (row < row1) {
                const __nv_bfloat16 *x = row < p.Hq ? q + row * p.sq.h : k + (row - p.Hq) * p.sk.h;
                xa[u] = *reinterpret_cast<const uint2 *>(x + ch.a);
                xb[u] = *reinterpret_cast<const uint2 *>(x + ch.b);
            }
        }
    };
    load(row0);
    if (threadIdx.x < static_cast<unsigned>(p.rot >> 1)) 
        angle(p, position(p, b, l), turns_per_token(p, threadIdx.x), threadIdx.x, tab);
    uint2 wq[2], wk[2];  // as bf16: as fp32 they cost a block of the SM's five
    if constexpr (NORM) {
        wq[0] = *reinterpret_cast<const uint2 *>(p.wq + ch.a), wq[1] = *reinterpret_cast<const uint2 *>(p.wq + ch.b);
        wk[0] = *reinterpret_cast<const uint2 *>(p.wk + ch.a), wk[1] = *reinterpret_cast<const uint2 *>(p.wk + ch.b);
    }
    __syncthreads();
    Factors<D, INTER> f;
    if (ch.turns) f.load(tab, lane);
    for (int base = row0; base < row1; base += kAhead * kSlots) {
        if (base > row0) load(base);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int row = base + slot + u * kSlots;
            if (base + u * kSlots >= row1) break;  // block-uniform
            Eight y = unpack(xa[u], xb[u]);
            if constexpr (NORM) {
                float2 ss = mul2(y.v[0], y.v[0]);
#pragma unroll
                for (int e = 1; e < 4; ++e) ss = fma2(y.v[e], y.v[e], ss);
                const float r = rsqrtf(row_sum<LPR>(ss.x + ss.y) * (1.f / D) + p.eps);
                const float2 r2 = make_float2(r, r);
                const bool isq = row < p.Hq;
                const Eight w = unpack(isq ? wq[0] : wk[0], isq ? wq[1] : wk[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) y.v[e] = mul2(y.v[e], mul2(r2, w.v[e]));
            }
            if (ch.turns) f.rotate(y);
            if (row < row1) store_eight(row < p.Hq ? qo + row * p.sqo.h : ko + (row - p.Hq) * p.sko.h, ch, y);
        }
    }
}

// Gradient with norms: a block walks its own run of tokens, so that the weight's
// gradient gathers in registers over all of its rows; one partial sum per block, added
// up in block order by the second kernel (the same order every time).
// A block takes query rows only or key rows only, in proportion to their rounds: the
// weight is the block's, not the row's.  A slot (the lanes of a row) keeps one token of
// a group and takes its heads kHeads apart, kRows of them in a round, so the angles
// stay in its registers over the group's rounds and its pointers move by constant
// strides; other head counts than multiples of 8 leave slots idle in the last round.
// The next group's angles are computed while this one's rows are, one a thread, between
// two barriers.  Rows are copied to shared memory kAhead rounds before they are needed.
// Latency bounds it (0.57 instructions a scheduler and cycle, fixed latencies the first
// stall, DRAM at 41 %), which fewer instructions shorten: 4 x 2047 tokens of 24 heads took 44 us
// with the rows dealt to the slots in order and a channel's partner in another lane (337
// instructions a warp for two rows), 39 with pairs in a lane and fixed tokens (204), 37
// with 2 blocks of 102 registers an SM instead of 3 of 80 (169), and takes 35 with two
// rows a round (153); the 151 MB would take 23.
constexpr int kHeads = 4;
constexpr int kRows = 2;
constexpr int kAhead = 2;
constexpr int kRingBytes = (kAhead + 1) * kRows * 2 * kThreads * 16;

// (Nothing is read at `src` where the row is not `in`: zeros are written.)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// A block of query rows (ISQ) or of key rows: its `block` of the kind's `blocks`.  (The
// kind is a template's so that strides and weights are the launch's constants: chosen
// at run time they cost 40 integer instructions a round.)
template <int D, bool INTER, bool ISQ>
__device__ __forceinline__ void backward_block(const Params &p, int block, int blocks) {
    constexpr int LPR = D / 8, kSlots = kThreads / LPR, kTokens = kSlots / kHeads;
    static_assert(kTokens * (D / 2) == kThreads, "an angle a thread");
    __shared__ __align__(16) Table<D> tab[2][kTokens];
    extern __shared__ uint4 dynamic[];
    __nv_bfloat16 *const ring = reinterpret_cast<__nv_bfloat16 *>(dynamic);  // [kAhead + 1][kRows][2][kSlots][D]
    float (*red)[D + 4] = reinterpret_cast<float (*)[D + 4]>(dynamic);       // [kSlots], after the last row
    static_assert(kSlots * (D + 4) * sizeof(float) <= kRingBytes, "the sums fit in the rows' place");
    const int heads = ISQ ? p.Hq : p.Hkv;
    const Strides &sx = ISQ ? p.sq : p.sk, &sg = ISQ ? p.sdq : p.sdk, &so = ISQ ? p.sqo : p.sko;
    const int n_tokens = p.B * p.L;
    const int t0 = static_cast<int>(static_cast<long long>(n_tokens) * block / blocks);
    const int t1 = static_cast<int>(static_cast<long long>(n_tokens) * (block + 1) / blocks);
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const int sub = slot / kHeads, h0 = slot % kHeads;
    const Channels ch(p, lane);
    grid_dep_wait();
    grid_dep_launch();
    const Eight w = load_eight(ISQ ? p.wq : p.wk, ch);
    Eight acc = {};

    // The places of token `group + of` of the groups one after the other: moves l and
    // returns the sequences that the move leaves behind.
    auto next_group = [&](int &l) {
        l += kTokens;
        int wraps = 0;
        while (l >= p.L) l -= p.L, ++wraps;
        return wraps;
    };
    auto move = [&](auto *&ptr, const Strides &s, int wraps) {
        ptr += kTokens * s.l;
        if (wraps) ptr += wraps * (s.b - p.L * s.l);
    };

    // this thread's pair and its token of the group, for the tables
    const int pair = threadIdx.x % (D / 2), pair_of = threadIdx.x / (D / 2);
    const double per_token = pair < (p.rot >> 1) ? turns_per_token(p, pair) : 0.;
    int pair_l = (t0 + pair_of) % p.L, pair_b = (t0 + pair_of) / p.L;
    auto angles = [&](int group, int buf) {
        if (group + pair_of < t1 && pair < (p.rot >> 1))
            angle(p, position(p, pair_b, pair_l), per_token, pair, tab[buf][pair_of]);
        pair_b += next_group(pair_l);
    };

    // A walk over the slot's rows: head h0 + round kHeads of token group + sub, at place l
    // of its sequence.  The loads' walk (in_) is kAhead rounds before the computation's.
    const int first_l = (t0 + sub) % p.L;
    const long long seq = (t0 + sub) / p.L;
    const __nv_bfloat16 *x0 = (ISQ ? p.q : p.k) + seq * sx.b + first_l * sx.l + h0 * sx.h + lane * 8, *xp = x0;
    const __nv_bfloat16 *g0 = (ISQ ? p.dq : p.dk) + seq * sg.b + first_l * sg.l + h0 * sg.h + lane * 8, *gp = g0;
    __nv_bfloat16 *o0 = (ISQ ? p.qo : p.ko) + seq * so.b + first_l * so.l + h0 * so.h;
    int in_group = t0, in_h = h0, in_l = first_l, out_l = first_l;
    uint32_t fill = smem_addr(dynamic) + threadIdx.x * 16;
    const uint32_t fill_end = fill + kRingBytes;
    auto fetch = [&]() {  // a round's rows
        if (in_group < t1) {
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const bool in = in_group + sub < t1 && in_h + u * kHeads < heads;
                copy16(fill + u * 2 * kThreads * 16, xp, in);
                copy16(fill + (u * 2 + 1) * kThreads * 16, gp, in);
                xp += kHeads * sx.h;
                gp += kHeads * sg.h;
            }
            in_h += kRows * kHeads;
            if (in_h - h0 >= heads) {
                in_h = h0;
                in_group += kTokens;
                const int wraps = next_group(in_l);
                move(x0, sx, wraps);
                move(g0, sg, wraps);
                xp = x0;
                gp = g0;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        fill += kRows * 2 * kThreads * 16;
        if (fill == fill_end) fill -= kRingBytes;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch();
    angles(t0, 0);
    __syncthreads();
    int take = 0;
    for (int group = t0, which = 0; group < t1; group += kTokens, which ^= 1) {
        if (group + kTokens < t1) angles(group + kTokens, which ^ 1);
        Factors<D, INTER> f;
        const bool token = group + sub < t1;
        if (ch.turns) f.load(tab[which][token ? sub : 0], lane);  // a slot without a token turns zeros
        __nv_bfloat16 *op = o0;
        for (int base = 0; base < heads; base += kRows * kHeads) {
            // the rows are there, all lanes' parts of them, and those before them are read
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            __syncwarp();
            fetch();
            const __nv_bfloat16 *row = ring + (take * kRows * 2 * kSlots + slot) * D;
            take = take == kAhead ? 0 : take + 1;
            Eight x[kRows], g[kRows], t[kRows];
            float sum[kRows], mean[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                x[u] = load_eight(row + u * 2 * kSlots * D, ch);
                g[u] = load_eight(row + (u * 2 + 1) * kSlots * D, ch);
                if (ch.turns) f.rotate(g[u]);
                float2 ss = mul2(x[u].v[0], x[u].v[0]), dot = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 1; e < 4; ++e) ss = fma2(x[u].v[e], x[u].v[e], ss);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    t[u].v[e] = mul2(g[u].v[e], w.v[e]);
                    dot = fma2(t[u].v[e], x[u].v[e], dot);
                }
                sum[u] = ss.x + ss.y;
                mean[u] = dot.x + dot.y;
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) row_sums<LPR>(sum[u], mean[u]);
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const bool in = token && base + u * kHeads + h0 < heads;
                const float r = rsqrtf(sum[u] * (1.f / D) + p.eps);
                const float rr = in ? r : 0.f;  // (a row past the last holds zeros, but eps may be 0)
                const float m = -mean[u] * r * r * (1.f / D);  // dx = r w g - h mean(w g h), h = x r
                const float2 r2 = make_float2(r, r), rr2 = make_float2(rr, rr), m2 = make_float2(m, m);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 hn = mul2(x[u].v[e], rr2);
                    acc.v[e] = fma2(g[u].v[e], hn, acc.v[e]);
                    t[u].v[e] = fma2(hn, m2, mul2(t[u].v[e], r2));
                }
                if (in) store_eight(op, ch, t[u]);
                op += kHeads * so.h;
            }
        }
        move(o0, so, next_group(out_l));
        __syncthreads();  // this table may be overwritten, the next one is there
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        red[slot][ch.a + 2 * e] = acc.v[e].x, red[slot][ch.a + 2 * e + 1] = acc.v[e].y;
        red[slot][ch.b + 2 * e] = acc.v[2 + e].x, red[slot][ch.b + 2 * e + 1] = acc.v[2 + e].y;
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) s += red[i][threadIdx.x];
        p.partial[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = s;
    }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) backward_kernel(const __grid_constant__ Params p) {
    const int block = blockIdx.x;
    if (block < p.q_blocks)
        backward_block<D, INTER, true>(p, block, p.q_blocks);
    else
        backward_block<D, INTER, false>(p, block - p.q_blocks, static_cast<int>(gridDim.x) - p.q_blocks);
}

// The weights' gradients: dwq sums partial[block][D] over the first q_blocks blocks,
// dwk over the others; 8 columns a block, 32 threads a column, always in the same order.
__global__ void __launch_bounds__(256) weight_kernel(const float *partial, int q_blocks, int blocks, int D, float *dwq,
                                                     float *dwk) {
    __shared__ float red[32][9];
    const int col = blockIdx.x * 8 + (threadIdx.x & 7), s = threadIdx.x >> 3;
    const bool isq = col < D;
    const int c = isq ? col : col - D, end = isq ? q_blocks : blocks;
    grid_dep_wait();
    grid_dep_launch();
    float sum = 0.f;
#pragma unroll 8
    for (int i = (isq ? 0 : q_blocks) + s; i < end; i += 32) sum += __ldcg(partial + static_cast<size_t>(i) * D + c);
    red[s][threadIdx.x & 7] = sum;
    __syncthreads();
    if (s == 0) {
#pragma unroll
        for (int i = 1; i < 32; ++i) sum += red[i][threadIdx.x & 7];
        (isq ? dwq : dwk)[c] = sum;
    }
}

int check(const Params &p, int D) {
    if (p.Hq < 1 || p.Hkv < 1) return TFA_ERR_HEADS;
    if (p.B < 1 || p.L < 1 || static_cast<long long>(p.B) * p.L > (1ll << 30) || p.Hq > (1 << 16) ||
        p.Hkv > (1 << 16))
        return TFA_ERR_SHAPE;
    // an output whose rows are one and the same place (an expanded tensor)
    if ((p.B > 1 && (!p.sqo.b || !p.sko.b)) || (p.L > 1 && (!p.sqo.l || !p.sko.l)) || (p.Hq > 1 && !p.sqo.h) ||
        (p.Hkv > 1 && !p.sko.h))
        return TFA_ERR_SHAPE;
    if (D != 64 && D != 128) return TFA_ERR_HEAD_DIM;
    if (p.rot < 0 || p.rot > D || p.rot % 16 != 0 || !std::isfinite(p.eps) || p.eps < 0.f || !std::isfinite(p.mscale))
        return TFA_ERR_ROPE;
    if (p.rot > 0 && !p.inv_freq) return TFA_ERR_NULL;
    if ((p.wq == nullptr) != (p.wk == nullptr)) return TFA_ERR_NULL;
    return TFA_OK;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool aligned(const Strides &s) { return s.b % 8 == 0 && s.l % 8 == 0 && s.h % 8 == 0; }
// (A dimension of size 1 has a stride that no address uses, which may be anything.)
Strides strides(const long long *s, int B, int L, int H) {
    return Strides{B > 1 ? s[0] : 0, L > 1 ? s[1] : 0, H > 1 ? s[2] : 0};
}

int launch_forward(Params &p, int D, cudaStream_t stream) {
    const int n_rows = p.Hq + p.Hkv, slots = kThreads / (D / 8);
    const int tokens = p.B * p.L;
    // A block takes all of a token's rows, so that its angles are computed once,
    // unless that leaves SMs without a block (decoding): then one round of rows.
    p.rows_per_block = tokens >= 4 * kSms ? n_rows : slots;
    const dim3 grid(tokens, (n_rows + p.rows_per_block - 1) / p.rows_per_block);
    const bool norm = p.wq != nullptr;
    using Kern = void (*)(Params);
    auto pick = [&](bool inter) -> Kern {
        if (D == 128)
            return norm ? (inter ? forward_kernel<128, true, true> : forward_kernel<128, true, false>)
                        : (inter ? forward_kernel<128, false, true> : forward_kernel<128, false, false>);
        return norm ? (inter ? forward_kernel<64, true, true> : forward_kernel<64, true, false>)
                    : (inter ? forward_kernel<64, false, true> : forward_kernel<64, false, false>);
    };
    const cudaError_t e = launch_after(pick(p.inter != 0), grid, kThreads, 0, stream, p);
    return e == cudaSuccess ? TFA_OK : report_cuda("qk_norm_rope launch", e);
}

int launch_backward(Params &p, int D, float *dwq, float *dwk, cudaStream_t stream) {
    const int tokens = p.B * p.L;
    // blocks in proportion to the rounds, one of each kind at least, none without a token
    constexpr int kRound = kRows * kHeads;
    const int rq = (p.Hq + kRound - 1) / kRound, rk = (p.Hkv + kRound - 1) / kRound;
    p.q_blocks = static_cast<int>(static_cast<long long>(kBwdBlocks) * rq / (rq + rk));
    p.q_blocks = p.q_blocks < 1 ? 1 : p.q_blocks > kBwdBlocks - 1 ? kBwdBlocks - 1 : p.q_blocks;
    int k_blocks = kBwdBlocks - p.q_blocks;
    if (p.q_blocks > tokens) p.q_blocks = tokens;
    if (k_blocks > tokens) k_blocks = tokens;
    const int blocks = p.q_blocks + k_blocks;
    using Kern = void (*)(Params);
    const Kern kern = D == 128 ? (p.inter ? backward_kernel<128, true> : backward_kernel<128, false>)
                               : (p.inter ? backward_kernel<64, true> : backward_kernel<64, false>);
    static std::atomic<bool> prepared[kMaxDevices][4];  // the attribute holds for one device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return report_cuda("cudaGetDevice", e);
    if (dev < 0 || dev >= kMaxDevices) return report_cuda("device index", cudaErrorInvalidDevice);
    std::atomic<bool> &ready = prepared[dev][(D == 128 ? 2 : 0) + (p.inter ? 1 : 0)];
    if (!ready.load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
        if (e != cudaSuccess) return report_cuda("cudaFuncSetAttribute(norm gradient smem)", e);
        ready.store(true, std::memory_order_release);
    }
    e = launch_after(kern, blocks, kThreads, kRingBytes, stream, p);
    if (e != cudaSuccess) return report_cuda("qk_norm_rope gradient launch", e);
    e = launch_after(weight_kernel, 2 * D / 8, 256, 0, stream, p.partial, p.q_blocks, blocks, D, dwq, dwk);
    return e == cudaSuccess ? TFA_OK : report_cuda("norm weight gradient launch", e);
}

}  // namespace rope
}  // namespace tfa

using tfa::rope::aligned;
using tfa::rope::strides;

extern "C" int tfa_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out, const long long *strd,
                                const void *q_weight, const void *k_weight, const double *inv_freq,
                                const int *positions, int positions_per_row, int first_position, int B, int L, int Hq,
                                int Hkv, int D, int rot, int interleaved, float eps, float mscale,
                                tfa_stream_t stream) {
    if (!q || !k || !q_out || !k_out || !strd) return TFA_ERR_NULL;
    tfa::rope::Params p = {};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.qo = static_cast<__nv_bfloat16 *>(q_out);
    p.ko = static_cast<__nv_bfloat16 *>(k_out);
    p.sq = strides(strd, B, L, Hq);
    p.sk = strides(strd + 3, B, L, Hkv);
    p.sqo = strides(strd + 6, B, L, Hq);
    p.sko = strides(strd + 9, B, L, Hkv);
    p.wq = static_cast<const __nv_bfloat16 *>(q_weight);
    p.wk = static_cast<const __nv_bfloat16 *>(k_weight);
    p.inv_freq = inv_freq;
    p.pos = positions;
    p.pos_per_row = positions_per_row;
    p.pos0 = first_position;
    p.B = B;
    p.L = L;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.rot = rot;
    p.eps = eps;
    p.mscale = mscale;
    p.inter = interleaved ? 1 : 0;
    if (const int rc = tfa::rope::check(p, D)) return rc;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(q_weight, 16) ||
        !aligned(k_weight, 16) || !aligned(inv_freq, 8) || !aligned(positions, 4) || !aligned(p.sq) ||
        !aligned(p.sk) || !aligned(p.sqo) || !aligned(p.sko))
        return TFA_ERR_ALIGN;
    return tfa::rope::launch_forward(p, D, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t tfa_qk_norm_rope_workspace(int D) {
    return static_cast<size_t>(tfa::rope::kBwdBlocks) * (D < 0 ? 0 : D) * sizeof(float);
}

extern "C" int tfa_qk_norm_rope_backward(const void *dq_out, const void *dk_out, const void *q, const void *k,
                                         void *dq, void *dk, float *dq_weight, float *dk_weight,
                                         const long long *strd, const void *q_weight, const void *k_weight,
                                         const double *inv_freq, const int *positions, int positions_per_row,
                                         int first_position, int B, int L, int Hq, int Hkv, int D, int rot,
                                         int interleaved, float eps, float mscale, void *workspace,
                                         tfa_stream_t stream) {
    if (!dq_out || !dk_out || !dq || !dk || !strd) return TFA_ERR_NULL;
    const bool norm = q_weight && k_weight;
    if (norm && (!q || !k || !dq_weight || !dk_weight || !workspace)) return TFA_ERR_NULL;
    tfa::rope::Params p = {};
    // without norms the gradient is the rotation back, the forward's kernel on dq_out and dk_out
    p.q = static_cast<const __nv_bfloat16 *>(norm ? q : dq_out);
    p.k = static_cast<const __nv_bfloat16 *>(norm ? k : dk_out);
    p.dq = static_cast<const __nv_bfloat16 *>(dq_out);
    p.dk = static_cast<const __nv_bfloat16 *>(dk_out);
    p.qo = static_cast<__nv_bfloat16 *>(dq);
    p.ko = static_cast<__nv_bfloat16 *>(dk);
    p.sdq = strides(strd, B, L, Hq);
    p.sdk = strides(strd + 3, B, L, Hkv);
    p.sq = norm ? strides(strd + 6, B, L, Hq) : p.sdq;
    p.sk = norm ? strides(strd + 9, B, L, Hkv) : p.sdk;
    p.sqo = strides(strd + 12, B, L, Hq);
    p.sko = strides(strd + 15, B, L, Hkv);
    p.wq = static_cast<const __nv_bfloat16 *>(q_weight);
    p.wk = static_cast<const __nv_bfloat16 *>(k_weight);
    p.inv_freq = inv_freq;
    p.pos = positions;
    p.pos_per_row = positions_per_row;
    p.pos0 = first_position;
    p.B = B;
    p.L = L;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.rot = rot;
    p.eps = eps;
    p.mscale = mscale;
    p.inter = interleaved ? 1 : 0;
    p.conj = 1;
    p.partial = static_cast<float *>(workspace);
    if (const int rc = tfa::rope::check(p, D)) return rc;
    if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(dq_out, 16) || !aligned(dk_out, 16) || !aligned(dq, 16) ||
        !aligned(dk, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(inv_freq, 8) ||
        !aligned(positions, 4) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(workspace, 4) ||
        !aligned(p.sq) || !aligned(p.sk) || !aligned(p.sdq) || !aligned(p.sdk) || !aligned(p.sqo) || !aligned(p.sko))
        return TFA_ERR_ALIGN;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return norm ? tfa::rope::launch_backward(p, D, dq_weight, dk_weight, s) : tfa::rope::launch_forward(p, D, s);
}
