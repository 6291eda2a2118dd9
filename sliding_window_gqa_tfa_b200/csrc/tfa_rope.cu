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

// cos and sin (times mscale) of pair i's angle at a position.
__device__ __forceinline__ float2 angle(const Params &p, int pos, int i) {
    constexpr double kInv2Pi = 0.15915494309189533577;
    double turns = static_cast<double>(pos) * p.inv_freq[i] * kInv2Pi;
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * static_cast<float>(turns), &s, &c);
    return make_float2(c * p.mscale, (p.conj ? -s : s) * p.mscale);
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

// The lane's cos / sin factors: half layout, 8 pairs; interleaved, 4.
template <bool INTER>
struct Factors {
    float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
    __device__ __forceinline__ void load(const float2 *tab, int lane8, int rot) {
        const int half = rot >> 4;  // lanes of a half (half layout)
        if (lane8 * 8 >= rot) {
#pragma unroll
            for (int e = 0; e < (INTER ? 4 : 8); ++e) c[e] = 1.f, s[e] = 0.f;
            return;
        }
        const int i0 = INTER ? lane8 * 4 : (lane8 < half ? lane8 : lane8 - half) * 8;
#pragma unroll
        for (int e = 0; e < (INTER ? 4 : 8); ++e) {
            const float2 t = tab[i0 + e];
            c[e] = t.x;
            // the first of a pair takes - sin, the second + sin
            s[e] = INTER ? t.y : (lane8 < half ? -t.y : t.y);
        }
    }
    // Rotates the lane's 8 channels; every lane of the warp calls it (the half
    // layout's partners sit rot / 16 lanes away).
    __device__ __forceinline__ void rotate(float (&y)[8], int lane8, int rot) const {
        if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = y[2 * e], b = y[2 * e + 1];
                y[2 * e] = fmaf(a, c[e], -b * s[e]);
                y[2 * e + 1] = fmaf(b, c[e], a * s[e]);
            }
        } else {
            const int half = rot >> 4;
            const int lane = threadIdx.x & 31;
            const int partner = lane8 * 8 >= rot ? lane : (lane8 < half ? lane + half : lane - half);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float o = __shfl_sync(0xffffffffu, y[e], partner);
                y[e] = fmaf(y[e], c[e], o * s[e]);
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

template <int D, bool NORM, bool INTER>
__global__ void __launch_bounds__(kThreads) forward_kernel(const __grid_constant__ Params p) {
    constexpr int LPR = D / 8, kSlots = kThreads / LPR;
    __shared__ float2 tab[D / 2];
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
    if (threadIdx.x < static_cast<unsigned>(p.rot >> 1)) tab[threadIdx.x] = angle(p, position(p, b, l), threadIdx.x);
    float wq[8], wk[8];
    if constexpr (NORM) {
        unpack(*reinterpret_cast<const uint4 *>(p.wq + lane8 * 8), wq);
        unpack(*reinterpret_cast<const uint4 *>(p.wk + lane8 * 8), wk);
    }
    __syncthreads();
    Factors<INTER> f;
    f.load(tab, lane8, p.rot);
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
            f.rotate(y, lane8, p.rot);
            if (row < row1)
                *reinterpret_cast<uint4 *>(row < p.Hq ? qo + row * p.sqo.h : ko + (row - p.Hq) * p.sko.h) = pack(y);
        }
    }
}

// Gradient with norms: blocks walk groups of tokens, so that the weight's gradient
// gathers in registers over all of a block's rows; one partial sum per block, added
// up in block order by the second kernel (the same order every time).
// A block takes query rows only or key rows only, in proportion to their heads: the
// strides and the tensors are then the same for all its threads, and a thread keeps
// one weight and one sum (with both kinds in a block the loop spilled and took 39
// instructions a channel).  With few heads a round holds several tokens' rows.
// The loads of a round are issued while the round before is computed, and the next
// tokens' angles while these ones' rows are.
constexpr int kMaxTokens = 4;  // tokens of a group

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) backward_kernel(const __grid_constant__ Params p) {
    constexpr int LPR = D / 8, kSlots = kThreads / LPR;
    __shared__ float2 tab[2][kMaxTokens][D / 2];
    __shared__ float red[kSlots][D + 4];
    const bool isq = static_cast<int>(blockIdx.x) < p.q_blocks;  // the block's kind
    const int block = isq ? blockIdx.x : blockIdx.x - p.q_blocks;
    const int blocks = isq ? p.q_blocks : static_cast<int>(gridDim.x) - p.q_blocks;
    const int heads = isq ? p.Hq : p.Hkv;
    const __nv_bfloat16 *xs = isq ? p.q : p.k, *gs = isq ? p.dq : p.dk;
    __nv_bfloat16 *os = isq ? p.qo : p.ko;
    const Strides sx = isq ? p.sq : p.sk, sg = isq ? p.sdq : p.sdk, so = isq ? p.sqo : p.sko;
    const int n_tokens = p.B * p.L;
    const int per = heads < kSlots ? min(kMaxTokens, kSlots / heads) : 1;  // tokens of a group
    const int rounds = (heads + kSlots - 1) / kSlots;
    const int n_groups = (n_tokens + per - 1) / per;
    const int lane8 = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const int sub = per > 1 ? slot / heads : 0, h0 = per > 1 ? slot - sub * heads : slot;  // (sub may be past the group)
    float w[8], acc[8];
    unpack(*reinterpret_cast<const uint4 *>((isq ? p.wq : p.wk) + lane8 * 8), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    // Every thread's token moves by the same number of tokens from group to group:
    // db sequences and dl rows, and where that leaves the sequence one more sequence
    // and L rows back.  Pointers move by the same, without a product or a division.
    const int stride = blocks * per, db = stride / p.L, dl = stride - db * p.L;
    struct Place {
        int t, b, l;
    };
    auto place = [&](int t) { return Place{t, t / p.L, t - t / p.L * p.L}; };
    auto move = [&](Place &c) {  // whether it left its sequence
        c.t += stride;
        c.b += db;
        c.l += dl;
        const bool wrap = c.l >= p.L;
        if (wrap) c.b += 1, c.l -= p.L;
        return wrap;
    };
    // the angles of a group's tokens, D / 2 threads a token
    Place at = place(block * per + threadIdx.x / (D / 2));
    const int pair = threadIdx.x % (D / 2);
    const bool fills = static_cast<int>(threadIdx.x) / (D / 2) < per && pair < (p.rot >> 1);
    auto angles = [&](int buf) {
        if (fills && at.t < n_tokens) tab[buf][threadIdx.x / (D / 2)][pair] = angle(p, position(p, at.b, at.l), pair);
        move(at);
    };
    const bool has = sub < per && h0 < heads;  // the slot has a row in a group's first round
    Place c = place(block * per + sub);
    const __nv_bfloat16 *xp = xs + c.b * sx.b + c.l * sx.l + h0 * sx.h + lane8 * 8;
    const __nv_bfloat16 *gp = gs + c.b * sg.b + c.l * sg.l + h0 * sg.h + lane8 * 8;
    __nv_bfloat16 *op = os + c.b * so.b + c.l * so.l + h0 * so.h + lane8 * 8;
    const long long mx = db * sx.b + dl * sx.l, mg = db * sg.b + dl * sg.l, mo = db * so.b + dl * so.l;
    const long long wx = sx.b - p.L * sx.l, wg = sg.b - p.L * sg.l, wo = so.b - p.L * so.l;
    uint4 xv, gv;
    auto load = [&](bool in, long long x_off, long long g_off) {
        xv = gv = make_uint4(0u, 0u, 0u, 0u);
        if (in) {
            xv = *reinterpret_cast<const uint4 *>(xp + x_off);
            gv = *reinterpret_cast<const uint4 *>(gp + g_off);
        }
    };
    int which = 0;
    bool live = has && c.t < n_tokens;
    load(live, 0, 0);
    angles(0);
    __syncthreads();
    for (int group = block; group < n_groups; group += blocks, which ^= 1) {
        Factors<INTER> f;
        f.load(tab[which][sub < per ? sub : 0], lane8, p.rot);
        angles(which ^ 1);
        __nv_bfloat16 *orow = op;
        int h = h0;
        for (int i = 0; i < rounds; ++i, h += kSlots, orow += kSlots * so.h) {
            float x[8], g[8];
            unpack(xv, x);
            unpack(gv, g);
            const bool in = live;
            if (i + 1 < rounds) {
                live = in && h + kSlots < heads;
                load(live, (i + 1) * kSlots * sx.h, (i + 1) * kSlots * sg.h);
            } else {
                const bool wrap = move(c);
                xp += mx + (wrap ? wx : 0);
                gp += mg + (wrap ? wg : 0);
                op += mo + (wrap ? wo : 0);
                live = has && c.t < n_tokens;
                load(live, 0, 0);
            }
            f.rotate(g, lane8, p.rot);
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
            if (in) *reinterpret_cast<uint4 *>(orow) = pack(g);
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
// dwk over the others; 32 columns a block, 8 threads a column, always in the same order.
__global__ void __launch_bounds__(256) weight_kernel(const float *partial, int q_blocks, int blocks, int D, float *dwq,
                                                     float *dwk) {
    __shared__ float red[8][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), s = threadIdx.x >> 5;
    const bool isq = col < D;
    const int c = isq ? col : col - D, end = isq ? q_blocks : blocks;
    float sum = 0.f;
#pragma unroll 4
    for (int i = (isq ? 0 : q_blocks) + s; i < end; i += 8) sum += partial[static_cast<size_t>(i) * D + c];
    red[s][threadIdx.x & 31] = sum;
    __syncthreads();
    if (s == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) sum += red[i][threadIdx.x & 31];
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
    weight_kernel<<<2 * D / 32, 256, 0, stream>>>(p.partial, p.q_blocks, blocks, D, dwq, dwk);
    e = cudaGetLastError();
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
