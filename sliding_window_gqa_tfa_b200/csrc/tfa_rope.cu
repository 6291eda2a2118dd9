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
// Layout: a row is D / 8 lanes of 16 bytes, so a warp instruction moves whole
// 128-byte lines; tokens come in the projection's order ([B, L, H, D], any
// strides) and leave in the attention's ([B, H, L, D], or a cache's rows), so
// no separate transpose reads the data again.
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
constexpr int kBwdBlocks = 444;  // gradient kernel: most blocks, so most partial sums of a weight

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

__device__ __forceinline__ int position(const Params &p, int b, int l) {
    if (!p.pos) return p.pos0 + l;
    return p.pos_per_row ? __ldg(p.pos + static_cast<long long>(b) * p.L + l) : __ldg(p.pos + b) + l;
}

// What the channels of a position are multiplied by: each by its own c, its partner by
// its own s (minus the sine for a pair's first channel); channels past rot by 1 and 0.
// A lane's 8 channels lie as two float4, the lanes' first ones side by side, so that a
// row's lanes read different banks.
template <int D>
struct Table {
    float c[D], s[D];
    __device__ __forceinline__ static int at(int channel) {
        return ((channel >> 2) & 1) * (D / 2) + (channel >> 3) * 4 + (channel & 3);
    }
};

// Pair i's angle at a position, into its two channels.
template <int D>
__device__ __forceinline__ void angle(const Params &p, int pos, int i, Table<D> &tab) {
    constexpr double kInv2Pi = 0.15915494309189533577;
    double turns = static_cast<double>(pos) * p.inv_freq[i] * kInv2Pi;
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * static_cast<float>(turns), &s, &c);
    c *= p.mscale;
    s *= p.conj ? -p.mscale : p.mscale;
    const int a = p.inter ? 2 * i : i, b = p.inter ? 2 * i + 1 : i + (p.rot >> 1);
    tab.c[Table<D>::at(a)] = tab.c[Table<D>::at(b)] = c;
    tab.s[Table<D>::at(a)] = -s;
    tab.s[Table<D>::at(b)] = s;
}
// The channels that pass through.
template <int D>
__device__ __forceinline__ void pass_through(const Params &p, Table<D> &tab) {
    const int i = p.rot + threadIdx.x;
    if (i < D) tab.c[Table<D>::at(i)] = 1.f, tab.s[Table<D>::at(i)] = 0.f;
}

__device__ __forceinline__ void unpack(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The lane's 8 channels' factors; interleaved, one cosine and sine a pair.
template <int D, bool INTER>
struct Factors {
    float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
    __device__ __forceinline__ void load(const Table<D> &tab, int lane8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(tab.c + i * (D / 2) + lane8 * 4);
            const float4 y = *reinterpret_cast<const float4 *>(tab.s + i * (D / 2) + lane8 * 4);
            if constexpr (INTER) {
                c[2 * i] = x.x, c[2 * i + 1] = x.z;
                s[2 * i] = y.y, s[2 * i + 1] = y.w;
            } else {
                c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
                s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
            }
        }
    }
    // Rotates the lane's 8 channels; every lane of the warp calls it (the half
    // layout's partners sit in another lane: partner).
    __device__ __forceinline__ void rotate(float (&y)[8], int partner) const {
#pragma unroll
        for (int e = 0; e < (INTER ? 4 : 8); ++e) {
            if constexpr (INTER) {
                const float a = y[2 * e], b = y[2 * e + 1];
                y[2 * e] = fmaf(a, c[e], -b * s[e]);
                y[2 * e + 1] = fmaf(b, c[e], a * s[e]);
            } else {
                const float o = __shfl_sync(0xffffffffu, y[e], partner);
                y[e] = fmaf(y[e], c[e], o * s[e]);
            }
        }
    }
};
// The half layout's partner lane: rot / 16 lanes away, in the same row.
__device__ __forceinline__ int partner_lane(int lane8, int rot) {
    const int half = rot >> 4, lane = threadIdx.x & 31;
    return lane8 * 8 >= rot ? lane : (lane8 < half ? lane + half : lane - half);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int D, bool NORM, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) forward_kernel(const __grid_constant__ Params p) {
    constexpr int LPR = D / 8, kSlots = kThreads / LPR;
    __shared__ __align__(16) Table<D> tab;
    const int token = blockIdx.x, b = token / p.L, l = token - b * p.L;
    const int lane8 = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const int n_rows = p.Hq + p.Hkv;
    const int row0 = blockIdx.y * p.rows_per_block;
    const int row1 = min(row0 + p.rows_per_block, n_rows);
    const __nv_bfloat16 *q = p.q + b * p.sq.b + l * p.sq.l + lane8 * 8;
    const __nv_bfloat16 *k = p.k + b * p.sk.b + l * p.sk.l + lane8 * 8;
    __nv_bfloat16 *qo = p.qo + b * p.sqo.b + l * p.sqo.l + lane8 * 8;
    __nv_bfloat16 *ko = p.ko + b * p.sko.b + l * p.sko.l + lane8 * 8;
    // the first rows are on their way while the table is computed
    constexpr int kAhead = 4;
    uint4 x[kAhead];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int row = base + slot + u * kSlots;
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (row < row1)
                x[u] = *reinterpret_cast<const uint4 *>(row < p.Hq ? q + row * p.sq.h : k + (row - p.Hq) * p.sk.h);
        }
    };
    load(row0);
    if (threadIdx.x < static_cast<unsigned>(p.rot >> 1)) angle(p, position(p, b, l), threadIdx.x, tab);
    pass_through(p, tab);
    float wq[8], wk[8];
    if constexpr (NORM) {
        unpack(*reinterpret_cast<const uint4 *>(p.wq + lane8 * 8), wq);
        unpack(*reinterpret_cast<const uint4 *>(p.wk + lane8 * 8), wk);
    }
    __syncthreads();
    Factors<D, INTER> f;
    f.load(tab, lane8);
    const int partner = partner_lane(lane8, p.rot);
    for (int base = row0; base < row1; base += kAhead * kSlots) {
        if (base > row0) load(base);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int row = base + slot + u * kSlots;
            if (base + u * kSlots >= row1) break;  // block-uniform
            float y[8];
            unpack(x[u], y);
            if constexpr (NORM) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
                const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= r * (row < p.Hq ? wq[e] : wk[e]);
            }
            f.rotate(y, partner);
            if (row < row1)
                *reinterpret_cast<uint4 *>(row < p.Hq ? qo + row * p.sqo.h : ko + (row - p.Hq) * p.sko.h) = pack(y);
        }
    }
}

// Gradient with norms: a block walks its own run of tokens, so that the weight's
// gradient gathers in registers over all of its rows; one partial sum per block, added
// up in block order by the second kernel (the same order every time).
// A block takes query rows only or key rows only, in proportion to their heads: the
// strides and the tensors are then the same for all its threads, and a thread keeps
// one weight and one sum (with both kinds in a block the loop spilled and took 39
// instructions a channel).  The run's rows, token by token and head by head, are dealt
// to the slots (the lanes of a row) in turn; a slot's pointers move from row to row by
// constant strides.  The next row's loads are issued while a row is computed, and the
// angles of the next four tokens while these four's rows are, by all threads, between
// two barriers (a barrier and a fourth of the threads for each token: 50 us for 4 x
// 2047 tokens of 24 heads, this way BWD_US us; the 151 MB would take 23).
constexpr int kTokens = 4;  // of a table

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) backward_kernel(const __grid_constant__ Params p) {
    constexpr int LPR = D / 8, kSlots = kThreads / LPR;
    __shared__ __align__(16) Table<D> tab[2][kTokens];
    __shared__ float red[kSlots][D + 4];
    const bool isq = static_cast<int>(blockIdx.x) < p.q_blocks;  // the block's kind
    const int block = isq ? blockIdx.x : blockIdx.x - p.q_blocks;
    const int blocks = isq ? p.q_blocks : static_cast<int>(gridDim.x) - p.q_blocks;
    const int heads = isq ? p.Hq : p.Hkv;
    const Strides sx = isq ? p.sq : p.sk, sg = isq ? p.sdq : p.sdk, so = isq ? p.sqo : p.sko;
    const int n_tokens = p.B * p.L;
    const int t0 = static_cast<int>(static_cast<long long>(n_tokens) * block / blocks);
    const int t1 = static_cast<int>(static_cast<long long>(n_tokens) * (block + 1) / blocks);
    const int lane8 = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const int partner = partner_lane(lane8, p.rot);
    float w[8], acc[8];
    unpack(*reinterpret_cast<const uint4 *>((isq ? p.wq : p.wk) + lane8 * 8), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;

    // a table's angles: D / 2 threads a token, kThreads / (D / 2) tokens at a time
    auto angles = [&](int first, int buf) {
#pragma unroll
        for (int k = 0; k < kTokens; k += kThreads / (D / 2)) {
            const int sub = k + threadIdx.x / (D / 2), i = threadIdx.x % (D / 2), t = first + sub;
            if (sub < kTokens && t < t1 && i < (p.rot >> 1)) angle(p, position(p, t / p.L, t % p.L), i, tab[buf][sub]);
        }
    };
    for (int i = 0; i < 2 * kTokens; ++i) pass_through(p, tab[i / kTokens][i % kTokens]);

    // the slot's row: head h of token `sub` of the group, at place l of its sequence; a row
    // further is `dsub` tokens and `dh` heads further, and a token more where that passes
    // the last head
    const int dsub = kSlots / heads, dh = kSlots - dsub * heads;
    const int sub0 = slot / heads, h0 = slot - sub0 * heads;
    int l0 = (t0 + sub0) % p.L;  // of the group's first row
    const long long seq = (t0 + sub0) / p.L;
    const __nv_bfloat16 *x0 = (isq ? p.q : p.k) + seq * sx.b + l0 * sx.l + h0 * sx.h + lane8 * 8;
    const __nv_bfloat16 *g0 = (isq ? p.dq : p.dk) + seq * sg.b + l0 * sg.l + h0 * sg.h + lane8 * 8;
    __nv_bfloat16 *o0 = (isq ? p.qo : p.ko) + seq * so.b + l0 * so.l + h0 * so.h + lane8 * 8;
    const __nv_bfloat16 *xp, *gp;
    __nv_bfloat16 *op;
    int group = t0, rows = 0, row = 0, sub = 0, h = 0, l = 0;
    uint4 xv, gv;
    auto load = [&](bool in) {
        xv = gv = make_uint4(0u, 0u, 0u, 0u);
        if (in) {
            xv = *reinterpret_cast<const uint4 *>(xp);
            gv = *reinterpret_cast<const uint4 *>(gp);
        }
    };
    auto enter = [&]() {  // the first row of the group
        rows = min(kTokens, t1 - group) * heads;
        row = slot, sub = sub0, h = h0, l = l0, xp = x0, gp = g0, op = o0;
        load(row < rows);
    };
    auto next_row = [&]() {
        row += kSlots;
        sub += dsub;
        l += dsub;
        h += dh;
        xp += dsub * sx.l + dh * sx.h;
        gp += dsub * sg.l + dh * sg.h;
        op += dsub * so.l + dh * so.h;
        if (h >= heads) {
            h -= heads, sub += 1, l += 1;
            xp += sx.l - heads * sx.h;
            gp += sg.l - heads * sg.h;
            op += so.l - heads * so.h;
        }
        while (l >= p.L) {
            l -= p.L;
            xp += sx.b - p.L * sx.l;
            gp += sg.b - p.L * sg.l;
            op += so.b - p.L * so.l;
        }
        load(row < rows);
    };
    auto next_group = [&]() {
        group += kTokens;
        l0 += kTokens;
        x0 += kTokens * sx.l;
        g0 += kTokens * sg.l;
        o0 += kTokens * so.l;
        while (l0 >= p.L) {
            l0 -= p.L;
            x0 += sx.b - p.L * sx.l;
            g0 += sg.b - p.L * sg.l;
            o0 += so.b - p.L * so.l;
        }
        if (group < t1) enter();
    };

    grid_dep_launch();
    enter();
    angles(t0, 0);
    __syncthreads();
    for (int which = 0, here = t0; here < t1; here += kTokens, which ^= 1) {
        if (here + kTokens < t1) angles(here + kTokens, which ^ 1);
        const int n_rows = min(kTokens, t1 - here) * heads;
        for (int base = 0; base < n_rows; base += kSlots) {
            float x[8], g[8];
            unpack(xv, x);
            unpack(gv, g);
            const bool in = base + slot < n_rows;
            __nv_bfloat16 *const out = op;
            Factors<D, INTER> f;
            f.load(tab[which][in ? sub : 0], lane8);
            if (base + kSlots < n_rows) next_row();
            else next_group();
            f.rotate(g, partner);
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
            const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
            const float rr = in ? r : 0.f;  // (a row past the last holds zeros, but eps may be 0)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gx = g[e] * x[e];
                dot = fmaf(gx, w[e], dot);
                acc[e] = fmaf(gx, rr, acc[e]);
            }
            dot = row_sum<LPR>(dot);
            const float m = -dot * r * r * (1.f / D);  // dx = r (w g - x r^2 mean(w g x))
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = r * fmaf(x[e], m, g[e] * w[e]);
            if (in) *reinterpret_cast<uint4 *>(out) = pack(g);
        }
        __syncthreads();  // this table may be overwritten, the next one is there
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) red[slot][lane8 * 8 + e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) s += red[i][threadIdx.x];
        p.partial[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = s;
    }
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
    if (p.B < 1 || p.L < 1 || static_cast<long long>(p.B) * p.L > (1ll << 30) || p.Hq > (1 << 20) ||
        p.Hkv > (1 << 20))
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
Strides strides(const long long *s) { return Strides{s[0], s[1], s[2]}; }

int launch_forward(Params &p, int D, cudaStream_t stream) {
    const int n_rows = p.Hq + p.Hkv, slots = kThreads / (D / 8);
    const int tokens = p.B * p.L;
    // A block takes all of a token's rows, so that its angles are computed once,
    // unless that leaves SMs without a block (decoding): then one round of rows.
    p.rows_per_block = tokens >= 4 * 148 ? n_rows : slots;
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
    pick(p.inter != 0)<<<grid, kThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TFA_OK : report_cuda("qk_norm_rope launch", e);
}

int launch_backward(Params &p, int D, float *dwq, float *dwk, cudaStream_t stream) {
    const int tokens = p.B * p.L;
    // blocks in proportion to the heads, one of each kind at least, none without a token
    p.q_blocks = static_cast<int>(static_cast<long long>(kBwdBlocks) * p.Hq / (p.Hq + p.Hkv));
    p.q_blocks = p.q_blocks < 1 ? 1 : p.q_blocks > kBwdBlocks - 1 ? kBwdBlocks - 1 : p.q_blocks;
    int k_blocks = kBwdBlocks - p.q_blocks;
    if (p.q_blocks > tokens) p.q_blocks = tokens;
    if (k_blocks > tokens) k_blocks = tokens;
    const int blocks = p.q_blocks + k_blocks;
    using Kern = void (*)(Params);
    const Kern kern = D == 128 ? (p.inter ? backward_kernel<128, true> : backward_kernel<128, false>)
                               : (p.inter ? backward_kernel<64, true> : backward_kernel<64, false>);
    kern<<<blocks, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return report_cuda("qk_norm_rope gradient launch", e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * D / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];  // set up while the first kernel runs, which it waits for
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, weight_kernel, static_cast<const float *>(p.partial), p.q_blocks, blocks, D, dwq, dwk);
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
    p.sq = strides(strd);
    p.sk = strides(strd + 3);
    p.sqo = strides(strd + 6);
    p.sko = strides(strd + 9);
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
    p.sdq = strides(strd);
    p.sdk = strides(strd + 3);
    p.sq = norm ? strides(strd + 6) : p.sdq;
    p.sk = norm ? strides(strd + 9) : p.sdk;
    p.sqo = strides(strd + 12);
    p.sko = strides(strd + 15);
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
