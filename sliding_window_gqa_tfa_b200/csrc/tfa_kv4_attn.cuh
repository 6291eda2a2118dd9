// tfa_kv4_attn.cuh -- attention of few rows over the 4-bit cache.
//
// For a query row q of a KV group and cached position j, with s and m the step
// and minimum of a group of 32 channels and c its codes:
//   q.k_j = sum_groups [ s (sum_d q_d c_d) + m (sum_d q_d) ],
//   o     = sum_j p_j v_j = sum_j [ (p_j s) c_d + p_j m ]   per channel d,
// so the tensor core multiplies q and p s with the codes themselves, and K and V
// are never rounded.  A code in the low four bits of a 16-bit word is the
// subnormal c 2^-24 of fp16, one in the next four c 2^-20, both exact: a pair of
// codes costs one logical operation, and no offset has to come off again.  (As
// bf16, 0x4300 | c = 128 + c, the loop took 370 instructions for 16 positions
// instead of 250 and was bound by issuing them: 39 us for 16 sequences of at most
// 8192 positions; p s rounded to bf16 left an error of 0.0024 of the output
// instead of 0.0017.)
// fp16 needs its range kept:
//   q   is scaled by a power of two for each row, its largest magnitude just below
//       2^15: exact but for channels 2^-28 and more below the largest;
//   p   is taken against a reference r (in log2 units) with p s < 2^15, so r follows
//       the scores and the steps: terms down to 2^-30 of the largest survive the
//       rounding, 2^-11 relative above 2^-20.  r, not the maximum, is what pieces
//       are joined by.  Steps are taken to lie in [2^-40, 2^80] there.
// The minima's part of the scores is one more product, of the (s, m) words as they
// lie in the cache with (0, sum q), the sum split into two bf16.
//
// What bounds it is reading the cache (1.25 D bytes a position and head) as long
// as a group's rows are few, so the products are transposed: positions (K) and
// channels (V) are the 16-row side of mma.m16n8k16, the query rows its 8-column
// side, and eight rows cost what the codes need anyway.  Every warp walks its own
// 32-position steps with its own asynchronous copies and its own reference and
// sum; nothing in the loop waits for another warp.  The fragments come straight
// from the codes: a lane's word of 8 codes gives four fp16 pairs, in an order of
// channels that q is laid out in once.
//
// A segment is a sequence's KV head and a chunk of its rows.  Lengths are read on
// the device, where every CTA works out the same deal (Deal): longer sequences'
// segments are cut into more pieces, about as many pieces in all as there are
// CTAs, and a piece lies in one segment, since to start one (queries, first
// copies, the join of its warps) costs as much as some 25 steps.  A segment in one
// piece is finished there; the pieces of a cut one go to a workspace and are
// joined by a second kernel (r* = max r, l* = sum 2^(r - r*) l, likewise O).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <math_constants.h>

#include "tfa_ptx.cuh"

namespace tfa {
namespace kv4 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kStep = 32;      // positions of a warp's step
constexpr int kWarps = 4;      // of a CTA
constexpr int kMaxSeqs = 1024;  // sequences of a call
constexpr int kMaxRounds = 4;   // pieces of a CTA that cut segments may ask for

struct DecodeParams {
    const __nv_bfloat16 *q;  // [B, Hq, L, D]
    __nv_bfloat16 *o;        // [B, Hq, L, D]
    const uint8_t *kc, *vc;  // [B, Hkv, cap, D / 2]
    const uint32_t *km, *vm;  // [B, Hkv, cap, D / 32]
    const int *lens;          // [B], or nullptr: `all` positions each
    int all;
    const float *sinks;       // [Hq] or nullptr
    float *part;              // workspace: [kMaxRounds CTAs][rows (D + 2)], a slot a piece
    unsigned *status;
    int B, Hq, Hkv, L, G, cap;
    int rows;                 // G L: query rows of a KV head
    int chunks;               // of 8 NB rows
    int window, first;
    float scale, scale_log2, softcap;
};

// The steps of one sequence: the first `fs` cover the first tokens that stay
// visible, the others the window (or everything) from step fs + gap on.
struct Span {
    int n;      // cached positions
    int steps;  // in all
    int fs, gap;
};
__device__ __forceinline__ Span span_of(const DecodeParams &p, int n) {
    Span s;
    s.n = n < 0 || n > p.cap ? 0 : n;
    s.fs = s.gap = s.steps = 0;
    if (s.n == 0) return s;
    s.steps = (s.n + kStep - 1) / kStep;
    if (p.window > 0) {
        // 64 bits: a window may be as large as an int
        const long long lo = static_cast<long long>(s.n) - p.L - p.window + 1;  // first position in the window
        const int first_step = lo > 0 ? static_cast<int>(lo / kStep) : 0;
        const int keep = (min(p.first, s.n) + kStep - 1) / kStep;
        if (first_step > keep) {
            s.fs = keep;
            s.gap = first_step - keep;
            s.steps -= s.gap;
        }
    }
    return s;
}

// How the segments are cut: each segment of a sequence of n steps into
// k = ceil(n / T) pieces, T the least (about) for which the pieces do not pass the
// CTAs (or a small multiple of them, if the segments do; from kMaxRounds of them on
// nothing is cut).  Pieces are numbered by sequence, segment and place; CTA c takes
// c, c + grid, ..  Up to 32 sequences are held one per lane, the same in every warp;
// more in shared memory.  Every lane of a warp calls the members together.
struct Deal {
    int HC, B, lane;   // segments of a sequence
    int n, k, before;  // B <= 32: the lane's sequence: length, pieces of a segment, those of the sequences before
    int *first;        // B > 32: pieces of a segment before each sequence, [B + 1]
    int total;         // of all sequences, for one segment each
    float inv_t;

    __device__ __forceinline__ int pieces(int steps) const {
        return steps == 0 ? 0 : max(1, static_cast<int>(ceilf(steps * inv_t)));
    }
    __device__ __forceinline__ Deal(const DecodeParams &p, int grid, int *shared, bool report)
        : HC(p.Hkv * p.chunks), B(p.B), lane(threadIdx.x & 31), n(0), k(0), before(0), first(shared) {
        int *steps_of = shared + kMaxSeqs + 1;
        int mine = 0;
        float all = 0.f;
        int count = 0;
        if (B <= 32) {
            if (lane < B) n = p.lens ? load_input<true>(p.lens + lane) : p.all;
            if (report && threadIdx.x < 32 && (n < 0 || n > p.cap)) atomicOr(p.status, TFA_DEVICE_BAD_SEQLENS);
            mine = span_of(p, n).steps;
            count = __popc(__ballot_sync(0xffffffffu, mine > 0));
            all = static_cast<float>(mine);
        } else {
            for (int b = threadIdx.x; b < B; b += blockDim.x) {
                const int len = p.lens ? load_input<true>(p.lens + b) : p.all;
                if (report && (len < 0 || len > p.cap)) atomicOr(p.status, TFA_DEVICE_BAD_SEQLENS);
                steps_of[b] = span_of(p, len).steps;
            }
            __syncthreads();
            for (int b = lane; b < B; b += 32) {
                all += static_cast<float>(steps_of[b]);
                count += steps_of[b] > 0;
            }
            count = __reduce_add_sync(0xffffffffu, count);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
        const int rounds = min(kMaxRounds, max(1, (count * HC + grid - 1) / grid));
        const int most = max(count, rounds * grid / HC);  // pieces for one segment each
        float T = fmaxf(all / static_cast<float>(max(most, 1)), static_cast<float>(kWarps));
        for (int tries = 0; ; ++tries) {
            inv_t = tries < 16 ? 1.f / T : 0.f;  // (0: one piece a segment)
            int sum = 0;
            if (B <= 32) {
                k = pieces(mine);
                sum = k;
            } else {
                for (int b = lane; b < B; b += 32) sum += pieces(steps_of[b]);
            }
            total = __reduce_add_sync(0xffffffffu, sum);
            if (total <= most) break;
            T *= fmaxf(1.02f, static_cast<float>(total) / static_cast<float>(most));
        }
        if (B <= 32) {
            int incl = k;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            before = incl - k;
            return;
        }
        if (threadIdx.x < 32) {
            const int per = (B + 31) / 32, a0 = min(lane * per, B), a1 = min(a0 + per, B);
            int sum = 0;
            for (int i = a0; i < a1; ++i) sum += pieces(steps_of[i]);
            int incl = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            int run = incl - sum;
            for (int i = a0; i < a1; ++i) {
                first[i] = run;
                run += pieces(steps_of[i]);
            }
            if (lane == 31) first[B] = incl;
        }
        __syncthreads();
    }
    // The sequence that holds piece x < total HC: the last that begins at or before it.
    __device__ __forceinline__ int find(int x) const {
        if (B <= 32) return 31 - __clz(__ballot_sync(0xffffffffu, lane < B && before * HC <= x));
        int lo = 0, hi = B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] * HC <= x) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
    __device__ __forceinline__ int begin(int b) const {
        return (B <= 32 ? __shfl_sync(0xffffffffu, before, b) : first[b]) * HC;
    }
    __device__ __forceinline__ int pieces_of(int b) const {
        return B <= 32 ? __shfl_sync(0xffffffffu, k, b) : first[b + 1] - first[b];
    }
    __device__ __forceinline__ int length(const DecodeParams &p, int b) const {
        return B <= 32 ? __shfl_sync(0xffffffffu, n, b) : p.lens ? load_input<true>(p.lens + b) : p.all;
    }
};

// -------------------------------------------------------------- instructions
// d = a b + d, a b (d from zero), fp16; a b, bf16.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}
__device__ __forceinline__ void mma0_bf16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}
// Transpose of an 8 x 8 matrix of 16-bit words, a row's two words per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Codes i and i + 4 of a word (bits 4 i and 16 + 4 i) as an fp16 pair: c 2^-24 for
// even i, c 2^-20 for odd.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    return (w >> (I & 2 ? 8 : 0)) & (I & 1 ? 0x00f000f0u : 0x000f000fu);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, bool in) {
    const int n = in ? BYTES : 0;  // 0: the destination is filled with zeros
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
// A row's words of steps and minima.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
    else
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
}
// Four 8 x 8 matrices of 16-bit words, a row's address from each lane: lane (g, t)
// gets words 2 t, 2 t + 1 of row g (TRANS: of column g) of each.
template <bool TRANS>
__device__ __forceinline__ void load_matrices(uint32_t a, uint32_t (&w)[4]) {
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
}

// NB: blocks of 8 columns (query rows).  REP (NB = 1): with at most 8 / REP rows the
// columns hold REP copies of them, copy c for the groups g = c (mod REP): p times a
// step is then taken once for all of a product's columns, not once for each group
// (at REP = 4 a fifth of the instructions: 16 sequences of 2 rows 31 -> 27.7 us).
template <int D, int NB, int REP = 1>
struct Cfg {
    static_assert(NB == 1 || REP == 1, "copies fill one block of columns");
    static constexpr int kCols = 8 / REP;             // columns of a copy
    static constexpr int kParts = (D / 32) / REP;     // groups of a copy

    static constexpr int kGroups = D / 32;
    static constexpr int kRowBytes = D / 2, kMetaBytes = D / 8;
    static constexpr int kRows = 8 * NB;
    static constexpr int kCtasPerSm = NB == 1 ? 4 : 2;  // the register file
    static constexpr int kStages = (NB == 1 && D == 128) ? 2 : 4;  // what shared memory holds
    static constexpr int kHalfStage = kStep * (kRowBytes + kMetaBytes);  // K or V of a step
    static constexpr int kPipeBytes = kWarps * kStages * 2 * kHalfStage;
    static constexpr int kOutStride = D + 4;  // floats; the 4 keep the writes of a warp in different banks
    // joining the warps, over the pipeline's buffers: O, m and l of each
    static constexpr int kJoinBytes = kWarps * kRows * (kOutStride + 2) * 4;
    static constexpr int kSmemBytes = kPipeBytes > kJoinBytes ? kPipeBytes : kJoinBytes;
    static constexpr int kSlotFloats = kRows * (D + 2);
};

// Position of 16-byte chunk c (a group's codes) of row r: the chunks of eight rows
// then lie in different banks.
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
    return D == 128 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1);
}

// O += P V for a step's two 16-row tiles.  A group's 16 bytes are eight 16-bit words
// of four channels each: the transposing load hands lane (g, t) word g of rows 2 t and
// 2 t + 1, channels 32 gr + 4 g .. + 3 of two positions, as the product's A side takes
// them.  copy: of the lane's columns 2 t and 2 t + 1; part f of it is group f REP + copy.
// SAFE: a position that a row does not see adds nothing even where its step or
// minimum is not finite.
template <int D, int NB, int REP, bool SAFE>
__device__ __forceinline__ void add_values(float (&o)[D / 16][NB][4], float (&om)[D / 32 / REP][NB][2],
                                           const float (&pr)[2][NB][4], uint32_t vcodes, uint32_t vmeta,
                                           const uint32_t (&chunk)[D / 32], int g, int copy) {
    using C = Cfg<D, NB, REP>;
    uint32_t m0[2][C::kParts], m1[2][C::kParts];  // rows g and g + 8 of each tile
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
        const uint32_t row = vmeta + (16 * tile + g) * C::kMetaBytes;
        if constexpr (REP == 1) {
            lds_words(row, m0[tile]);
            lds_words(row + 8 * C::kMetaBytes, m1[tile]);
        } else {
#pragma unroll
            for (int f = 0; f < C::kParts; ++f) {
                m0[tile][f] = lds32(row + (f * REP + copy) * 4);
                m1[tile][f] = lds32(row + 8 * C::kMetaBytes + (f * REP + copy) * 4);
            }
        }
    }
#pragma unroll
    for (int f = 0; f < C::kParts; ++f) {
        uint32_t b[2][NB][2];
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
            const uint32_t x0 = m0[tile][f], x1 = m1[tile][f];
            const float s0 = __uint_as_float(x0 << 16), n0 = __uint_as_float(x0 & 0xffff0000u);
            const float s1 = __uint_as_float(x1 << 16), n1 = __uint_as_float(x1 & 0xffff0000u);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float *q = pr[tile][nb];
                auto times = [](float a, float b) { return SAFE && a == 0.f ? 0.f : a * b; };
                b[tile][nb][0] = transpose8(pack_f16(times(q[0], s0), times(q[1], s0)));
                b[tile][nb][1] = transpose8(pack_f16(times(q[2], s1), times(q[3], s1)));
                if (SAFE) {
                    om[f][nb][0] += times(q[0], n0) + times(q[2], n1);
                    om[f][nb][1] += times(q[1], n0) + times(q[3], n1);
                } else {
                    om[f][nb][0] = fmaf(q[2], n1, fmaf(q[0], n0, om[f][nb][0]));
                    om[f][nb][1] = fmaf(q[3], n1, fmaf(q[1], n0, om[f][nb][1]));
                }
            }
        }
#pragma unroll
        for (int c = 0; c < REP; ++c) {
            const int gr = f * REP + c;
            uint32_t w[4];
            load_matrices<true>(vcodes + chunk[gr], w);
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
                const uint32_t wa = w[2 * tile], wb = w[2 * tile + 1];
                const uint32_t a0[4] = {code_pair<0>(wa), code_pair<1>(wa), code_pair<0>(wb), code_pair<1>(wb)};
                const uint32_t a1[4] = {code_pair<2>(wa), code_pair<3>(wa), code_pair<2>(wb), code_pair<3>(wb)};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    mma(o[2 * gr][nb], a0, b[tile][nb]);
                    mma(o[2 * gr + 1][nb], a1, b[tile][nb]);
                }
            }
        }
    }
}

template <int D, int NB, int REP>
__global__ void __launch_bounds__(32 * kWarps, Cfg<D, NB, REP>::kCtasPerSm)
    decode_kernel(const __grid_constant__ DecodeParams p) {
    using C = Cfg<D, NB, REP>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int shared[2 * kMaxSeqs + 1];
    grid_dep_wait();
    grid_dep_launch();  // the joining kernel may be set up meanwhile; it waits for this one's end
    const Deal deal(p, gridDim.x, shared, blockIdx.x == 0);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int copy = 2 * t / C::kCols;  // of the lane's columns 2 t and 2 t + 1
    const uint32_t pipe = smem_addr(smem) + warp * C::kStages * 2 * C::kHalfStage;
    // where chunk gr of row `lane` lies: the address a lane gives to load_matrices
    uint32_t chunk[C::kGroups];
#pragma unroll
    for (int gr = 0; gr < C::kGroups; ++gr) chunk[gr] = lane * C::kRowBytes + chunk_at<D>(lane, gr) * 16;
    // chunk `lane` of a step's codes: row lane / (chunks a row), in that row's order
    const uint32_t copy_to = (lane / (C::kRowBytes / 16)) * C::kRowBytes +
                             chunk_at<D>(lane / (C::kRowBytes / 16), lane % (C::kRowBytes / 16)) * 16;
    float *jo = reinterpret_cast<float *>(smem);                      // [warp][row][kOutStride]
    float *jm = jo + kWarps * C::kRows * C::kOutStride, *jl = jm + kWarps * C::kRows;  // [warp][row]

    const int n_pieces = deal.total * deal.HC;
    for (int piece = blockIdx.x; piece < n_pieces; piece += gridDim.x) {
        const int b = deal.find(piece), cuts = deal.pieces_of(b);
        const Span sp = span_of(p, deal.length(p, b));
        const int rel = piece - deal.begin(b), hc = rel / cuts, place = rel - hc * cuts;
        const int each = sp.steps / cuts, more = sp.steps - each * cuts;  // the first `more` pieces take one more
        const int j0 = each * place + min(place, more), j1 = j0 + each + (place < more ? 1 : 0);
        const int h = hc / p.chunks, row0 = (hc - h * p.chunks) * C::kRows;
        const int n_rows = min(C::kRows, p.rows - row0);
        const size_t plane = (static_cast<size_t>(b) * p.Hkv + h) * p.cap;
        const size_t qrow = (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(h) * p.G) * p.L + row0;

        const int p0 = sp.n - p.L;  // position of the sequence's first new row
        // the last position that has left the last row's window (-1: none)
        const int past = p.window > 0 ? max(-1, sp.n - 1 - min(p.window, sp.n)) : -1;

        // the query rows, asked for ahead of the copies that all warps ask for at once
        uint4 qv[NB][C::kGroups];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int gr = 0; gr < C::kGroups; ++gr) {
                qv[nb][gr] = make_uint4(0u, 0u, 0u, 0u);
                const int row = 8 * nb + g % C::kCols;
                if (row < n_rows)
                    qv[nb][gr] = load_input<true>(reinterpret_cast<const uint4 *>(p.q + (qrow + row) * D + 32 * gr + 8 * t));
            }

        // copies of step j into stage st: codes in 16-byte chunks, steps and minima row by
        // row.  A lane's chunks lie 512 bytes apart on both sides (their rows' chunk
        // orders agree), so a whole step takes one address a tensor.
        const uint8_t *kc = p.kc + plane * C::kRowBytes + lane * 16, *vc = p.vc + plane * C::kRowBytes + lane * 16;
        const uint32_t *km = p.km + (plane + lane) * C::kGroups, *vm = p.vm + (plane + lane) * C::kGroups;
        auto issue = [&](int j, uint32_t base) {
            const int key0 = (j < sp.fs ? j : j + sp.gap) * kStep;
            constexpr int kChunks = C::kRowBytes / 16, kCopies = kStep * kChunks / 32;
            const size_t co = static_cast<size_t>(key0) * C::kRowBytes, mo = static_cast<size_t>(key0) * C::kGroups;
            const uint32_t dst = base + copy_to, mdst = base + kStep * C::kRowBytes + lane * C::kMetaBytes;
            if (key0 + kStep <= sp.n) {
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    cp_async<16>(dst + i * 512, kc + co + i * 512);
                    cp_async<16>(dst + C::kHalfStage + i * 512, vc + co + i * 512);
                }
                cp_async<C::kMetaBytes>(mdst, km + mo);
                cp_async<C::kMetaBytes>(mdst + C::kHalfStage, vm + mo);
            } else {  // the last step: rows past the end are filled with zeros, nothing is read
                const int left = sp.n - key0;
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const bool in = (i * 32 + lane) / kChunks < left;
                    cp_async<16>(dst + i * 512, kc + (in ? co + i * 512 : 0), in);
                    cp_async<16>(dst + C::kHalfStage + i * 512, vc + (in ? co + i * 512 : 0), in);
                }
                cp_async<C::kMetaBytes>(mdst, km + (lane < left ? mo : 0), lane < left);
                cp_async<C::kMetaBytes>(mdst + C::kHalfStage, vm + (lane < left ? mo : 0), lane < left);
            }
        };
#pragma unroll
        for (int st = 0; st < C::kStages - 1; ++st) {
            if (j0 + warp + st * kWarps < j1) issue(j0 + warp + st * kWarps, pipe + st * 2 * C::kHalfStage);
            cp_commit();
        }

        // the query rows as B fragments: lane (g, t) holds row g's channels 32 gr + 8 t ..
        // + 7, paired as the codes are (i, i + 4), those of odd i scaled by 2^-4 against
        // the codes' 2^4; bs: (0, sum of the group's q) of group t, split in two bf16;
        // unit: what makes log2 scores of the products, for rows 2 t and 2 t + 1
        uint32_t bq[NB][C::kGroups][2][2], bs[NB][2];
        float unit[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const uint4 (&v)[C::kGroups] = qv[nb];
            float top = 0.f, sum[C::kGroups];
#pragma unroll
            for (int gr = 0; gr < C::kGroups; ++gr) {
                const uint32_t w[4] = {v[gr].x, v[gr].y, v[gr].z, v[gr].w};
                sum[gr] = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = __uint_as_float(w[e] << 16), y = __uint_as_float(w[e] & 0xffff0000u);
                    top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
                    sum[gr] += x + y;
                }
                sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
                sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // rho = 2^(14 - e), 2^e the power of two at or below the row's largest
            const int e = max(-86, static_cast<int>(__float_as_uint(top) >> 23) - 127);
            const float size = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
            // a negative scale's sign goes with q, a scale of 0 makes it 0, so that the
            // unit is positive
            const float rho = p.scale > 0.f ? size : p.scale < 0.f ? -size : 0.f;
#pragma unroll
            for (int gr = 0; gr < C::kGroups; ++gr) {
                const uint32_t w[4] = {v[gr].x, v[gr].y, v[gr].z, v[gr].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // channels i and i + 4
                    const uint32_t lo = w[i >> 1], hi = w[2 + (i >> 1)];
                    const float f = i & 1 ? rho * 0.0625f : rho;
                    const float x = __uint_as_float(i & 1 ? lo & 0xffff0000u : lo << 16);
                    const float y = __uint_as_float(i & 1 ? hi & 0xffff0000u : hi << 16);
                    bq[nb][gr][i >> 1][i & 1] = pack_f16(x * f, y * f);
                }
            }
            float mine = 0.f;
#pragma unroll
            for (int gr = 0; gr < C::kGroups; ++gr) mine = t == gr ? sum[gr] : mine;
            mine *= rho * 0x1p-24f;  // the codes' unit
            const float head = __bfloat162float(__float2bfloat16_rn(mine));
            bs[nb][0] = pack_bf16(0.f, mine);
            bs[nb][1] = pack_bf16(0.f, mine - head);
            const float un = 0x1p24f / size * (p.softcap > 0.f || p.scale == 0.f ? 1.f : fabsf(p.scale_log2));
            unit[nb][0] = __shfl_sync(0xffffffffu, un, 8 * t);
            unit[nb][1] = __shfl_sync(0xffffffffu, un, 8 * t + 4);
        }

        float mul[NB][2];  // what is still to be multiplied into the scores
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) mul[nb][e] = p.softcap > 0.f ? 1.f : unit[nb][e];
        uint32_t highest = 0u;  // the largest step of V so far, as a bf16 pattern, and 2^es above it
        float es = -40.f;
        float o[D / 16][NB][4], om[C::kParts][NB][2], m[NB][2], l[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][nb][e] = 0.f;
#pragma unroll
            for (int f = 0; f < C::kParts; ++f) om[f][nb][0] = om[f][nb][1] = 0.f;
            m[nb][0] = m[nb][1] = -CUDART_INF_F;
            l[nb][0] = l[nb][1] = 0.f;
        }

        constexpr uint32_t kStageBytes = 2 * C::kHalfStage, kPipe = C::kStages * kStageBytes;
        uint32_t here = 0, fill = kPipe - kStageBytes;  // the stage read now, the one filled now
        for (int j = j0 + warp; j < j1; j += kWarps) {
            const int ahead = j + (C::kStages - 1) * kWarps;
            if (ahead < j1) issue(ahead, pipe + fill);
            cp_commit();
            cp_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t kcodes = pipe + here, kmeta = kcodes + kStep * C::kRowBytes;
            const uint32_t vcodes = kcodes + C::kHalfStage, vmeta = vcodes + kStep * C::kRowBytes;
            fill = here;
            here = here + kStageBytes == kPipe ? 0 : here + kStageBytes;
            const int key0 = (j < sp.fs ? j : j + sp.gap) * kStep;

            // scores: [tile][nb][(position g, rows 2t, 2t + 1), (position g + 8, ..)]
            float sc[2][NB][4];
            uint32_t k0[2][C::kGroups], k1[2][C::kGroups];
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
                lds_words(kmeta + (16 * tile + g) * C::kMetaBytes, k0[tile]);
                lds_words(kmeta + (16 * tile + g + 8) * C::kMetaBytes, k1[tile]);
            }
            {
                // minima: the (s, m) word of group t of each position as it lies there, twice
                uint32_t x[4];
                if constexpr (D == 128) {
                    load_matrices<false>(kmeta + lane * C::kMetaBytes, x);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = t < C::kGroups ? lds32(kmeta + (8 * i + g) * C::kMetaBytes + t * 4) : 0u;
                }
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    const uint32_t a[4] = {x[2 * tile], x[2 * tile + 1], x[2 * tile], x[2 * tile + 1]};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma0_bf16(sc[tile][nb], a, bs[nb]);
                }
            }
#pragma unroll
            for (int gr = 0; gr < C::kGroups; ++gr) {
                uint32_t w[4];  // word t of the group of positions g, g + 8, g + 16, g + 24
                load_matrices<false>(kcodes + chunk[gr], w);
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    const uint32_t w0 = w[2 * tile], w1 = w[2 * tile + 1];
                    const uint32_t a0[4] = {code_pair<0>(w0), code_pair<0>(w1), code_pair<1>(w0), code_pair<1>(w1)};
                    const uint32_t a1[4] = {code_pair<2>(w0), code_pair<2>(w1), code_pair<3>(w0), code_pair<3>(w1)};
                    const float s0 = __uint_as_float(k0[tile][gr] << 16), s1 = __uint_as_float(k1[tile][gr] << 16);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        float acc[4];
                        mma0(acc, a0, bq[nb][gr][0]);
                        mma(acc, a1, bq[nb][gr][1]);
                        sc[tile][nb][0] = fmaf(s0, acc[0], sc[tile][nb][0]);
                        sc[tile][nb][1] = fmaf(s0, acc[1], sc[tile][nb][1]);
                        sc[tile][nb][2] = fmaf(s1, acc[2], sc[tile][nb][2]);
                        sc[tile][nb][3] = fmaf(s1, acc[3], sc[tile][nb][3]);
                    }
                }
            }
            if (p.softcap > 0.f) {  // log2 scores at once; unit is the products' own
                const float u = fabsf(p.scale) / p.softcap, cap2 = p.softcap * kLog2e;
#pragma unroll
                for (int tile = 0; tile < 2; ++tile)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[tile][nb][e] = cap2 * tanhf(sc[tile][nb][e] * unit[nb][e & 1] * u);
            }
            // only steps at the causal edge, the tail or the window's edge hold hidden pairs
            const bool edge = key0 + kStep - 1 > p0 || (key0 <= past && key0 + kStep > p.first);
            if (edge) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int hi_k = p0 + (row0 + 8 * nb + (2 * t + e) % C::kCols) % p.L;
                        const long long lo_k = p.window > 0 ? static_cast<long long>(hi_k) - p.window + 1 : 0;
#pragma unroll
                        for (int tile = 0; tile < 2; ++tile)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int k = key0 + tile * 16 + g + 8 * half;
                                if (k > hi_k || (k < lo_k && k >= p.first)) sc[tile][nb][2 * half + e] = -CUDART_INF_F;
                            }
                    }
            }

            // a power of two above the steps of V's rows so far, a row a lane
            {
                uint32_t w[C::kGroups], high = 0u;
                lds_words(vmeta + lane * C::kMetaBytes, w);
                // a row that none of the queries sees bounds nothing
                if (edge && p.window > 0 && key0 + lane <= p0 - static_cast<long long>(p.window) && key0 + lane >= p.first) {
#pragma unroll
                    for (int gr = 0; gr < C::kGroups; ++gr) w[gr] = 0u;
                }
#pragma unroll
                for (int gr = 0; gr < C::kGroups; ++gr) high = max(high, w[gr] & 0x7fffu);
                if (__any_sync(0xffffffffu, high > highest)) {
                    high = 0u;  // without steps that are not finite: they bound nothing
#pragma unroll
                    for (int gr = 0; gr < C::kGroups; ++gr)
                        high = max(high, (w[gr] & 0x7fffu) < 0x7f80u ? w[gr] & 0x7fffu : 0u);
                    highest = max(highest, __reduce_max_sync(0xffffffffu, high) | 0x7fu);  // bf16 patterns are ordered
                    es = static_cast<float>(min(80, max(-40, static_cast<int>(highest >> 7) - 126)));  // step < 2^es
                }
            }
            // the reference r of a row: moved up when 2^(score - r) 2^es would pass 2^15
            bool grow = false;
            float top[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[nb][e] = fmax3(sc[0][nb][e], sc[0][nb][2 + e], fmaxf(sc[1][nb][e], sc[1][nb][2 + e]));
                    top[nb][e] = fmaf(top[nb][e], mul[nb][e], es);
                    grow |= top[nb][e] - m[nb][e] > 15.f;  // (false where both are -inf)
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[nb][e];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        x = fmaxf(x - 7.f, m[nb][e]);
                        const float f = m[nb][e] == -CUDART_INF_F ? 0.f : ex2(m[nb][e] - x);
                        m[nb][e] = x;
                        l[nb][e] *= f;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            o[i][nb][e] *= f;
                            o[i][nb][2 + e] *= f;
                        }
#pragma unroll
                        for (int i = 0; i < C::kParts; ++i) om[i][nb][e] *= f;
                    }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mm = m[nb][e] == -CUDART_INF_F ? 0.f : m[nb][e];
#pragma unroll
                    for (int tile = 0; tile < 2; ++tile) {
                        sc[tile][nb][e] = ex2(fmaf(sc[tile][nb][e], mul[nb][e], -mm));
                        sc[tile][nb][2 + e] = ex2(fmaf(sc[tile][nb][2 + e], mul[nb][e], -mm));
                        l[nb][e] += sc[tile][nb][e] + sc[tile][nb][2 + e];
                    }
                }
            if (edge) add_values<D, NB, REP, true>(o, om, sc, vcodes, vmeta, chunk, g, copy);
            else add_values<D, NB, REP, false>(o, om, sc, vcodes, vmeta, chunk, g, copy);
            __syncwarp();  // every lane has read the stage that the next copies fill
        }
        cp_wait<0>();

        // join the warps: sums over the lanes that share a row, then m, l and O to shared memory
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], x);
#pragma unroll
                    for (int f = 0; f < C::kParts; ++f) om[f][nb][e] += __shfl_xor_sync(0xffffffffu, om[f][nb][e], x);
                }
            }
        __syncthreads();  // every warp's copies have landed and been read
#pragma unroll
        for (int f = 0; f < C::kParts; ++f) {
            // the lane's columns hold its copy's group of part f
            float x[NB][8];
#pragma unroll
            for (int c = 0; c < REP; ++c)
                if (REP == 1 || copy == c) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[nb][e] = o[2 * (f * REP + c)][nb][e];
                            x[nb][4 + e] = o[2 * (f * REP + c) + 1][nb][e];
                        }
                }
            const int gr = f * REP + (REP == 1 ? 0 : copy);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 8 * nb + (2 * t + e) % C::kCols;
                    *reinterpret_cast<float4 *>(jo + (warp * C::kRows + row) * C::kOutStride + 32 * gr + 4 * g) =
                        make_float4(fmaf(x[nb][e], 0x1p24f, om[f][nb][e]), fmaf(x[nb][2 + e], 0x1p20f, om[f][nb][e]),
                                    fmaf(x[nb][4 + e], 0x1p24f, om[f][nb][e]),
                                    fmaf(x[nb][6 + e], 0x1p20f, om[f][nb][e]));  // out of the codes' units
                    if (f == 0 && g == 0 && copy == 0) {
                        jm[warp * C::kRows + row] = m[nb][e];
                        jl[warp * C::kRows + row] = l[nb][e];
                    }
                }
        }
        __syncthreads();
        float *slot = p.part + static_cast<size_t>(piece) * C::kSlotFloats;  // (only cut segments have one)
        for (int i = threadIdx.x; i < n_rows * (D / 4); i += 32 * kWarps) {
            const int row = i / (D / 4), c4 = i % (D / 4);
            float mx = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, jm[w * C::kRows + row]);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = jm[w * C::kRows + row];
                if (mw == -CUDART_INF_F) continue;  // a warp without a visible position
                const float f = ex2(mw - mx);
                const float4 v = *reinterpret_cast<const float4 *>(jo + (w * C::kRows + row) * C::kOutStride + 4 * c4);
                sum = fmaf(f, jl[w * C::kRows + row], sum);
                a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
            }
            if (cuts == 1) {
                if (p.sinks && mx > -CUDART_INF_F)
                    sum += ex2(fmaf(load_input<true>(p.sinks + h * p.G + (row0 + row) / p.L), kLog2e, -mx));
                const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
                *reinterpret_cast<uint2 *>(p.o + (qrow + row) * D + 4 * c4) =
                    make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
            } else {
                __stcg(reinterpret_cast<float4 *>(slot + row * D + 4 * c4), a);
                if (c4 == 0) {
                    __stcg(slot + C::kRows * D + row, mx);
                    __stcg(slot + C::kRows * (D + 1) + row, sum);
                }
            }
        }
        __syncthreads();  // before the next piece's copies
    }
}

// One row of a segment, from its `cuts` pieces (0: zeros): a block's WARPS warps take
// the pieces in turn, a lane D / 32 channels; eight pieces' loads of each warp are in
// flight together.  Few rows may have as many pieces as there are CTAs (74 a segment
// for 8 segments): 16 warps ask for them all at once (1 x 32768 positions of 8 heads 19.7 -> 18.8 us); many rows have few
// pieces each, and blocks of 4 warps join more of them side by side.
template <int WARPS>
struct JoinShared {
    float o[WARPS][128], m[WARPS], l[WARPS];
};

template <int D, int NB, int WARPS>
__device__ __forceinline__ void join_row(const DecodeParams &p, JoinShared<WARPS> &sh, const float *slot0, int cuts, int row,
                                         int head, __nv_bfloat16 *out) {
    using C = Cfg<D, NB>;
    constexpr int kVec = D / 32, kBatch = 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float mx = -CUDART_INF_F, sum = 0.f, a[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) a[i] = 0.f;
    for (int k0 = warp; k0 < cuts; k0 += WARPS * kBatch) {
        float mk[kBatch], lk[kBatch], v[kBatch][kVec];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int k = k0 + u * WARPS;
            const float *s = slot0 + static_cast<size_t>(min(k, cuts - 1)) * C::kSlotFloats;
            mk[u] = k < cuts ? __ldcg(s + C::kRows * D + row) : -CUDART_INF_F;
            lk[u] = __ldcg(s + C::kRows * (D + 1) + row);
            const float *src = s + row * D + lane * kVec;
            if constexpr (kVec == 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
                v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
            } else {
                const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
                v[u][0] = x.x, v[u][1] = x.y;
            }
        }
        float mn = mx;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) mn = fmaxf(mn, mk[u]);
        const float f0 = mx == -CUDART_INF_F ? 0.f : ex2(mx - mn);
        sum *= f0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) a[i] *= f0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (mk[u] == -CUDART_INF_F) continue;
            const float f = ex2(mk[u] - mn);
            sum = fmaf(f, lk[u], sum);
#pragma unroll
            for (int i = 0; i < kVec; ++i) a[i] = fmaf(f, v[u][i], a[i]);
        }
        mx = mn;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) sh.o[warp][lane * kVec + i] = a[i];
    if (lane == 0) sh.m[warp] = mx, sh.l[warp] = sum;
    __syncthreads();
    if (threadIdx.x < D / 2) {
        mx = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, sh.m[w]);
        float x = 0.f, y = 0.f;
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (sh.m[w] == -CUDART_INF_F) continue;
            const float f = ex2(sh.m[w] - mx);
            sum = fmaf(f, sh.l[w], sum);
            x = fmaf(f, sh.o[w][2 * threadIdx.x], x);
            y = fmaf(f, sh.o[w][2 * threadIdx.x + 1], y);
        }
        if (p.sinks && mx > -CUDART_INF_F) sum += ex2(fmaf(load_input<true>(p.sinks + head), kLog2e, -mx));
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        reinterpret_cast<uint32_t *>(out)[threadIdx.x] = pack_bf16(x * inv, y * inv);
    }
    __syncthreads();
}

// Joins the pieces of the segments that were cut, row by row, and writes zeros for a
// sequence without a position.  Few blocks, each working out the deal once: they can
// be there before the main kernel ends.
template <int D, int NB, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) join_kernel(const __grid_constant__ DecodeParams p, int grid, int rows) {
    using C = Cfg<D, NB>;
    __shared__ int shared[2 * kMaxSeqs + 1];
    __shared__ JoinShared<WARPS> sh;
    // the lengths are there: the main kernel lets this one start after its own wait
    const Deal deal(p, grid, shared, false);
    grid_dep_wait();
    grid_dep_launch();
    for (int item = blockIdx.x; item < p.B * deal.HC * rows; item += gridDim.x) {
        const int segment = item / rows, row = item - segment * rows;
        const int b = segment / deal.HC, hc = segment - b * deal.HC;
        const int h = hc / p.chunks, first = (hc - h * p.chunks) * C::kRows + row;  // the row among the KV head's
        const int cuts = deal.pieces_of(b);  // 0: a sequence without a position
        if (first >= p.rows || cuts == 1) continue;  // (one piece: finished where it was computed)
        const size_t at = (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(h) * p.G) * p.L + first;
        join_row<D, NB, WARPS>(p, sh, p.part + static_cast<size_t>(deal.begin(b) + hc * cuts) * C::kSlotFloats, cuts, row,
                        h * p.G + first / p.L, p.o + at * D);
    }
}

}  // namespace kv4
}  // namespace tfa
