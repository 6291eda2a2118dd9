// tfa_kv4.cu -- a key/value cache held in 4 bits: writing rows into it, reading
// them back, and attention over it.
//
// Format, per cached position and KV head: D channels in groups of 32.  A group
// holds its minimum m and step s = bf16((max - m) / 15), and per channel the code
// c = rint((x - m) / s) in 0..15; the value is c s + m.  Codes: D / 2 bytes, byte
// i channel 2i (low half) and 2i + 1; steps and minima: one 32-bit word per
// group, s in the low half.  A group that holds a value that is not finite (or
// whose range is not) has s = m = NaN: it reads back as NaN.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "../../include/tfa.h"
#include "tfa_internal.h"
#include "tfa_kv4_attn.cuh"
#include "tfa_ptx.cuh"

namespace tfa {
namespace kv4 {

constexpr int kGroup = 32;  // channels that share a step and a minimum

struct Cache {
    uint8_t *kc, *vc;   // [B, Hkv, cap, D / 2]
    uint32_t *km, *vm;  // [B, Hkv, cap, D / 32]
};

// ------------------------------------------------------------ append and read
// n / d for n < 2^31 by a product: q = n m >> (31 + s), m = ceil(2^(31 + s) / d),
// s = ceil(log2 d) (m d - 2^(31 + s) < d <= 2^s bounds the error below 1 / d).
struct Divisor {
    unsigned d, m, s;
    __device__ __forceinline__ unsigned of(unsigned n) const {
        return static_cast<unsigned>((static_cast<unsigned long long>(n) * m) >> (31 + s));
    }
};
Divisor divisor(unsigned d) {
    Divisor r{d, 0u, 0u};
    while ((1ull << r.s) < d) ++r.s;
    r.m = static_cast<unsigned>(((1ull << (31 + r.s)) + d - 1) / d);
    return r;
}

struct AppendParams {
    const __nv_bfloat16 *k, *v;
    long long sk[3], sv[3];  // element strides over (batch, head, row)
    Cache c;
    const int *start;  // first cache row of each sequence; NULL: start0
    int start0;
    unsigned n_rows;  // B Hkv L
    Divisor L, Hkv;
    int cap;
    unsigned *status;
};

// Both kernels: a lane takes 16 channels of K and of V, half a group, so a row is
// D / 16 lanes.  They should be bound by the bytes moved (2.625 a channel each); what
// is measured is the wait for loads (append: 0.61 instructions a scheduler and cycle),
// which is short with few instructions beside (4 x 2047 rows of 8 heads, append and read: 49.6 us
// with 64-bit row indexes and IEEE divisions for the codes, 22.2 us without, 18.5 us
// with K and V found at once and packed arithmetic; the 88 MB would take 13.4).
// The codes of a lane's 16 channels, a and b, and the word of the step and minimum of
// the group that it shares with the lane beside it; every lane of the warp calls it.
__device__ __forceinline__ unsigned long long encode(const uint4 &a, const uint4 &b, uint32_t &meta) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    // extremes two by two, NaN if any value is
    auto h2 = [](uint32_t x) { return *reinterpret_cast<__nv_bfloat162 *>(&x); };
    __nv_bfloat162 mn = h2(w[0]), mx = mn;
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        mn = __hmin2_nan(mn, h2(w[e]));
        mx = __hmax2_nan(mx, h2(w[e]));
    }
    mn = __hmin2_nan(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
    mx = __hmax2_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    const float lo = __bfloat162float(__hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn)));
    const float hi = __bfloat162float(__hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx)));
    const float step = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(hi - lo, 15.f)));
    const bool fine = step <= 3.3895314e38f;  // false for NaN, and infinite with an infinite value or range
    // The codes: rint((x - lo) / step), ties to even.  The quotient is at most 15.06
    // (the step's own rounding), so no code passes 15.  One correction of the product
    // with the reciprocal makes every tie, a quotient of 5 bits, exact; adding 2^23
    // then rounds it, and the sum's low bits are the code.
    unsigned long long code = 0ull;
    auto value = [&](int e) {
        return (e & 1 ? __uint_as_float(w[e >> 1] & 0xffff0000u) : __uint_as_float(w[e >> 1] << 16)) - lo;
    };
    if (fine && step >= 0x1p-100f && step <= 0x1p100f) {
        const float inv = __frcp_rn(step);
        const float2 inv2 = make_float2(inv, inv), step2 = make_float2(-step, -step), lo2 = make_float2(-lo, -lo);
        uint32_t half[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            half[j] = 0u;
#pragma unroll
            for (int e = 3; e >= 0; --e) {
                const uint32_t x = w[4 * j + e];
                const float2 d = add2(make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), lo2);
                const float2 t = mul2(d, inv2);
                const float2 q = add2(fma2(fma2(t, step2, d), inv2, t), make_float2(8388608.f, 8388608.f));
                half[j] = (half[j] << 4) + __float_as_uint(q.y);
                half[j] = (half[j] << 4) + __float_as_uint(q.x);
            }
            half[j] -= 0xfb000000u;  // what the eight 0x4b000000 add up to: 0x4b000000 (1 + 16 + ...) mod 2^32
        }
        code = half[0] | static_cast<unsigned long long>(half[1]) << 32;
    } else if (fine && step > 0.f) {  // where the reciprocal or the correction could leave fp32's range
#pragma unroll
        for (int e = 0; e < 16; ++e)
            code |= static_cast<unsigned long long>(fminf(rintf(__fdiv_rn(value(e), step)), 15.f)) << (4 * e);
    }
    meta = fine ? (__float_as_uint(step) >> 16) | (__float_as_uint(lo) & 0xffff0000u) : 0x7fc07fc0u;
    return code;
}

template <int D>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int LPR = D / 16;
    const unsigned row = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int lane = threadIdx.x % LPR;
    const bool in = row < p.n_rows;
    const unsigned bh = in ? p.L.of(row) : 0u, i = in ? row - bh * p.L.d : 0u;
    const unsigned b = p.Hkv.of(bh), h = bh - b * p.Hkv.d;
    grid_dep_wait();
    grid_dep_launch();
    uint4 k[2] = {}, v[2] = {};
    if (in) {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.k + b * p.sk[0] + h * p.sk[1] + i * p.sk[2] + lane * 16);
        k[0] = src[0];
        k[1] = src[1];
        src = reinterpret_cast<const uint4 *>(p.v + b * p.sv[0] + h * p.sv[1] + i * p.sv[2] + lane * 16);
        v[0] = src[0];
        v[1] = src[1];
    }
    const long long first = p.start ? load_input<true>(p.start + b) : p.start0;
    uint32_t km, vm;
    const unsigned long long kc = encode(k[0], k[1], km), vc = encode(v[0], v[1], vm);
    if (!in || first < 0) return;  // a sequence without a place takes nothing
    const long long at = first + i;
    if (at >= p.cap) {
        if (lane == 0) atomicOr(p.status, TFA_DEVICE_BAD_SEQLENS);
        return;
    }
    const size_t dst = static_cast<size_t>(bh) * p.cap + at;
    reinterpret_cast<unsigned long long *>(p.c.kc)[dst * LPR + lane] = kc;
    reinterpret_cast<unsigned long long *>(p.c.vc)[dst * LPR + lane] = vc;
    if ((lane & 1) == 0) {
        p.c.km[dst * (D / kGroup) + lane / 2] = km;
        p.c.vm[dst * (D / kGroup) + lane / 2] = vm;
    }
}

struct ReadParams {
    Cache c;
    __nv_bfloat16 *k, *v;  // [B, Hkv, rows, D]
    const int *start;
    int start0;
    unsigned n_rows;  // B Hkv rows
    Divisor rows, Hkv;
    int cap;
    int split, skip;  // rows from `split` on lie `skip` cached positions further
    unsigned *status;
};

// Eight values from a word of codes; a code in the low bits of 0x4b000000 is 2^23 + c.
__device__ __forceinline__ uint4 values8(uint32_t code, float s, float m) {
    const uint32_t even = code & 0x0f0f0f0fu, odd = (code >> 4) & 0x0f0f0f0fu;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = __uint_as_float(__byte_perm(even, 0x4b000000u, 0x7440 + e)) - 8388608.f;
        const float b = __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7440 + e)) - 8388608.f;
        w[e] = pack_bf16(fmaf(a, s, m), fmaf(b, s, m));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// (A lane takes 8 channels here, so that a warp's store is one run of 512 bytes.)
template <int D>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int LPR = D / 8;
    const unsigned row = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int lane = threadIdx.x % LPR;
    const unsigned bh = p.rows.of(row), b = p.Hkv.of(bh);
    const int i = static_cast<int>(row - bh * p.rows.d);
    grid_dep_wait();
    grid_dep_launch();
    if (row >= p.n_rows) return;
    const long long first = p.start ? load_input<true>(p.start + b) : p.start0;
    const long long at = first + i + (i >= p.split ? p.skip : 0);
    uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
    if (first >= 0 && at < p.cap) {
        const size_t src = static_cast<size_t>(bh) * p.cap + at, code = src * LPR + lane, word = src * (D / kGroup) + lane / 4;
        const uint32_t kc = load_input<true>(reinterpret_cast<const uint32_t *>(p.c.kc) + code), km = load_input<true>(p.c.km + word);
        const uint32_t vc = load_input<true>(reinterpret_cast<const uint32_t *>(p.c.vc) + code), vm = load_input<true>(p.c.vm + word);
        k = values8(kc, __uint_as_float(km << 16), __uint_as_float(km & 0xffff0000u));
        v = values8(vc, __uint_as_float(vm << 16), __uint_as_float(vm & 0xffff0000u));
    } else if (first >= 0 && lane == 0) {
        atomicOr(p.status, TFA_DEVICE_BAD_SEQLENS);
    }
    const size_t dst = static_cast<size_t>(row) * LPR + lane;
    reinterpret_cast<uint4 *>(p.k)[dst] = k;
    reinterpret_cast<uint4 *>(p.v)[dst] = v;
}

// --------------------------------------------------------------- host checks
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_cache(const void *kc, const void *km, const void *vc, const void *vm, int B, int Hkv, int cap, int D) {
    if (!kc || !km || !vc || !vm) return TFA_ERR_NULL;
    if (Hkv < 1) return TFA_ERR_HEADS;
    if (B < 1 || cap < 1 || cap > (1 << 30) || static_cast<long long>(B) * Hkv * cap > (1ll << 40)) return TFA_ERR_SHAPE;
    if (D != 64 && D != 128) return TFA_ERR_HEAD_DIM;
    if (!aligned(kc, 16) || !aligned(km, 16) || !aligned(vc, 16) || !aligned(vm, 16)) return TFA_ERR_ALIGN;
    return TFA_OK;
}

// Blocks of 256 threads for `rows` rows of D / 16 lanes; 0 if there are more than
// 2^31 - 1 rows, counting those past the last in its block.
unsigned row_blocks(long long rows, int D) {
    return rows <= 0x7fffffffll - 256 ? static_cast<unsigned>((rows * (D / 16) + 255) / 256) : 0u;
}

int launch_read(const ReadParams &p, unsigned blocks, int D, cudaStream_t s) {
    // twice an append's lanes a row
    const cudaError_t e = launch_after(D == 128 ? read_kernel<128> : read_kernel<64>, 2 * blocks, 256, 0, s, p);
    return e == cudaSuccess ? TFA_OK : report_cuda("kv4 read launch", e);
}

// The cached positions that some of the last L rows sees: [0, keep) and [lo, S).
struct Seen {
    int keep, lo, rest;  // rest = S - lo
    long long rows() const { return static_cast<long long>(keep) + rest; }
};
Seen seen(int L, int S, int window, int first) {
    Seen r{0, 0, S};
    if (window > 0) {
        const long long lo = static_cast<long long>(S) - L - window + 1;
        const int keep = first < S ? first : S;
        if (lo > keep) r = Seen{keep, static_cast<int>(lo), S - static_cast<int>(lo)};
    }
    return r;
}

Cache cache_of(void *kc, void *km, void *vc, void *vm) {
    return Cache{static_cast<uint8_t *>(kc), static_cast<uint8_t *>(vc), static_cast<uint32_t *>(km),
                 static_cast<uint32_t *>(vm)};
}

// ------------------------------------------------------------------- decoding
constexpr int kMaxCtas = 640;  // of NB = 1, half of it of NB = 2: bounds the workspace whatever the device

template <int D, int NB, int REP>
int launch_decode(DecodeParams &p, int sms, cudaStream_t stream) {
    using C = Cfg<D, NB, REP>;
    p.chunks = (p.rows + C::kRows - 1) / C::kRows;
    static std::atomic<bool> prepared[kMaxDevices];  // the attribute holds for one device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return report_cuda("cudaGetDevice", e);
    if (!prepared[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(decode_kernel<D, NB, REP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return report_cuda("cudaFuncSetAttribute(kv4 decode smem)", e);
        prepared[dev].store(true, std::memory_order_release);
    }
    const int grid = sms * C::kCtasPerSm < kMaxCtas / NB ? sms * C::kCtasPerSm : kMaxCtas / NB;
    e = launch_after(decode_kernel<D, NB, REP>, grid, 32 * kWarps, C::kSmemBytes, stream, p);
    if (e != cudaSuccess) return report_cuda("kv4 decode launch", e);
    const int rows = p.chunks > 1 ? C::kRows : p.rows;
    const int items = p.B * p.Hkv * p.chunks * rows;
    const int warps = grid >= 32 * p.B * p.Hkv * p.chunks ? 16 : 4;  // 32 pieces of a segment or more: join_row
    e = launch_after(warps == 16 ? join_kernel<D, NB, 16> : join_kernel<D, NB, 4>, items < 4 * sms ? items : 4 * sms,
                     32 * warps, 0, stream, p, grid, rows);
    if (e != cudaSuccess)
        return report_cuda("kv4 join launch", e);
    return TFA_OK;
}

}  // namespace kv4
}  // namespace tfa

using namespace tfa::kv4;

extern "C" int tfa_kv4_append(const void *k, const void *v, const long long *strides, void *k_codes, void *k_meta,
                              void *v_codes, void *v_meta, const int *start, int first_row, int B, int Hkv, int L,
                              int capacity, int D, tfa_stream_t stream) {
    if (!k || !v || !strides) return TFA_ERR_NULL;
    if (int rc = check_cache(k_codes, k_meta, v_codes, v_meta, B, Hkv, capacity, D)) return rc;
    if (L < 1) return TFA_ERR_SHAPE;
    if (!start && (first_row < 0 || static_cast<long long>(first_row) + L > capacity)) return TFA_ERR_CACHE;
    AppendParams p = {};
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    const int sizes[3] = {B, Hkv, L};
    for (int i = 0; i < 3; ++i) {  // (a dimension of size 1 has a stride that no address uses)
        p.sk[i] = sizes[i] > 1 ? strides[i] : 0;
        p.sv[i] = sizes[i] > 1 ? strides[3 + i] : 0;
        if (p.sk[i] % 8 || p.sv[i] % 8) return TFA_ERR_ALIGN;
    }
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4)) return TFA_ERR_ALIGN;
    const unsigned blocks = row_blocks(static_cast<long long>(B) * Hkv * L, D);
    if (!blocks) return TFA_ERR_SHAPE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int sms = 0;
    if (int rc = tfa::device_info(s, &p.status, &sms)) return rc;
    p.c = cache_of(k_codes, k_meta, v_codes, v_meta);
    p.start = start;
    p.start0 = first_row;
    p.n_rows = static_cast<unsigned>(B) * Hkv * L;
    p.Hkv = divisor(Hkv);
    p.L = divisor(L);
    p.cap = capacity;
    const cudaError_t e = tfa::launch_after(D == 128 ? append_kernel<128> : append_kernel<64>, blocks, 256, 0, s, p);
    return e == cudaSuccess ? TFA_OK : tfa::report_cuda("kv4 append launch", e);
}

extern "C" int tfa_kv4_read(const void *k_codes, const void *k_meta, const void *v_codes, const void *v_meta, void *k,
                            void *v, const int *start, int first_row, int B, int Hkv, int rows, int capacity, int D,
                            tfa_stream_t stream) {
    if (!k || !v) return TFA_ERR_NULL;
    if (int rc = check_cache(k_codes, k_meta, v_codes, v_meta, B, Hkv, capacity, D)) return rc;
    if (rows < 1) return TFA_ERR_SHAPE;
    if (!start && (first_row < 0 || static_cast<long long>(first_row) + rows > capacity)) return TFA_ERR_CACHE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4)) return TFA_ERR_ALIGN;
    const unsigned blocks = row_blocks(static_cast<long long>(B) * Hkv * rows, D);
    if (!blocks) return TFA_ERR_SHAPE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ReadParams p = {};
    int sms = 0;
    if (int rc = tfa::device_info(s, &p.status, &sms)) return rc;
    p.c = cache_of(const_cast<void *>(k_codes), const_cast<void *>(k_meta), const_cast<void *>(v_codes),
                   const_cast<void *>(v_meta));
    p.k = static_cast<__nv_bfloat16 *>(k);
    p.v = static_cast<__nv_bfloat16 *>(v);
    p.start = start;
    p.start0 = first_row;
    p.n_rows = static_cast<unsigned>(B) * Hkv * rows;
    p.Hkv = divisor(Hkv);
    p.rows = divisor(rows);
    p.cap = capacity;
    p.split = rows;
    return launch_read(p, blocks, D, s);
}

namespace {

// a slot of 8 rows (NB = 1; 16 and half as many CTAs for NB = 2) for each piece of a cut segment
size_t decode_workspace(int D) { return static_cast<size_t>(kMaxRounds) * kMaxCtas * 8 * (D + 2) * sizeof(float); }

// The kernel for few rows, arguments checked: lens on the device, or `all` positions each.
int decode(const void *q, const void *k_codes, const void *k_meta, const void *v_codes, const void *v_meta,
           const int *lens, int all, void *o, int B, int Hq, int Hkv, int L, int capacity, int D, float scale,
           int window, int first, float softcap, const float *sinks, void *workspace, cudaStream_t s) {
    DecodeParams p = {};
    int sms = 0;
    if (int rc = tfa::device_info(s, &p.status, &sms)) return rc;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.kc = static_cast<const uint8_t *>(k_codes);
    p.vc = static_cast<const uint8_t *>(v_codes);
    p.km = static_cast<const uint32_t *>(k_meta);
    p.vm = static_cast<const uint32_t *>(v_meta);
    p.lens = lens;
    p.all = all;
    p.sinks = sinks;
    p.part = static_cast<float *>(workspace);
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.L = L;
    p.G = Hq / Hkv;
    p.cap = capacity;
    p.rows = p.G * L;
    p.window = window > 0 ? window : 0;
    p.first = first;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.softcap = softcap;
    if (D == 128)
        return p.rows <= 2   ? launch_decode<128, 1, 4>(p, sms, s)
               : p.rows <= 4 ? launch_decode<128, 1, 2>(p, sms, s)
               : p.rows <= 8 ? launch_decode<128, 1, 1>(p, sms, s)
                             : launch_decode<128, 2, 1>(p, sms, s);
    return p.rows <= 4   ? launch_decode<64, 1, 2>(p, sms, s)
           : p.rows <= 8 ? launch_decode<64, 1, 1>(p, sms, s)
                         : launch_decode<64, 2, 1>(p, sms, s);
}

// Whether a chunk goes to the kernel for few rows, which multiplies the codes as they
// are but walks them once for every 16 rows of a KV head, or is unpacked for the dense
// kernel: by estimates of both, in us.  The first spends a start for each piece (16 rows
// of a KV head; 2 blocks an SM) and a time for each of its rows and positions; the other
// the read back, and its key tiles in rounds of the SMs, or cut over all of them with a
// join.  Fitted to 1,181 sizes (D = 64 and 128, 1 to 16 heads a KV head, 1 to 8 KV heads,
// 1 to 16 sequences, 1 to 1,200 rows over 21 to 14,000 positions, windows of 1,024): the
// rule took the faster one or came within 15 % of it at 1,127, at most 2.3 times off
// (1,065 and 4.0 with a rule of the rows and of the products alone).  E.g. (D = 128) 128
// rows a KV head, one sequence of 5000: 28 against 76 us; 16 sequences: 270 against 160
// us; 200 rows of one head over 12000 positions: 18 against 446 us; 210 rows on 4 KV heads
// of 16 sequences of 159: 48 against 16 us.  (The SMs are those of a B200, not the
// device's count: tfa_kv4_prefill_workspace, which follows the rule, knows no device.)
bool few_rows(int B, int Hq, int Hkv, int L, int D, const Seen &sn) {
    const int G = Hq / Hkv;
    const long long rows = static_cast<long long>(G) * L;
    if (B > kMaxSeqs || static_cast<long long>(B) * Hq * L > (1ll << 26)) return false;
    if (rows <= 8) return true;  // its narrow form, always ahead
    const double d = D / 128., n = static_cast<double>(sn.rows()), heads = static_cast<double>(B) * Hkv;
    const double pieces = heads * static_cast<double>((rows + 15) / 16);
    const double own = 9 + (4.5 + 4.8 * d) * pieces / (2 * tfa::kSms) + (0.8 + 2.4 * d) * 16e-6 * pieces * n;
    const bool packed = L <= 128;  // several heads' rows in a tile
    const int per = L < 128 ? 128 / L : 1;
    const double items = packed ? heads * ((G + per - 1) / per) : heads * G * ((L + 255) / 256);
    const double tiles = std::ceil(n / 128), step = 1.3 + 0.8 * d, start = packed ? 11.5 : 16;
    const double whole = start + step * tiles * std::ceil(items / tfa::kSms);
    const double others = tfa::kSms / items < tiles ? tfa::kSms / items : tiles;  // pieces of a cut item
    const double cut = start + 8 + step * items * tiles / tfa::kSms + 3 * others;
    const double dense = (items < 4 * tfa::kSms && cut < whole ? cut : whole) + 0.9e-6 * heads * n * D;
    return own < 1.1 * dense;
}

}  // namespace

extern "C" size_t tfa_kv4_decode_workspace(int Hq, int Hkv, int L, int D) {
    return Hkv < 1 || Hq < 1 || L < 1 || D < 1 ? 0 : decode_workspace(D);
}

extern "C" int tfa_kv4_decode(const void *q, const void *k_codes, const void *k_meta, const void *v_codes,
                              const void *v_meta, const int *lens, void *o, int B, int Hq, int Hkv, int L,
                              int capacity, int D, float scale, int window, int first, float softcap,
                              const float *sinks, void *workspace, tfa_stream_t stream) {
    if (!q || !o || !lens || !workspace) return TFA_ERR_NULL;
    if (int rc = check_cache(k_codes, k_meta, v_codes, v_meta, B, Hkv, capacity, D)) return rc;
    if (Hq < 1 || Hq % Hkv != 0) return TFA_ERR_HEADS;
    if (B > kMaxSeqs || L < 1 || L > TFA_MAX_DECODE_ROWS || static_cast<long long>(B) * Hq * L > (1ll << 26))
        return TFA_ERR_SHAPE;
    if (first < 0 || (first > 0 && window <= 0)) return TFA_ERR_WINDOW;
    if (!std::isfinite(scale)) return TFA_ERR_SCALE;
    if (!std::isfinite(softcap) || softcap < 0.f || (softcap > 0.f && scale == 0.f)) return TFA_ERR_SOFTCAP;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lens, 4) || !aligned(sinks, 4) || !aligned(workspace, 16))
        return TFA_ERR_ALIGN;
    return decode(q, k_codes, k_meta, v_codes, v_meta, lens, 0, o, B, Hq, Hkv, L, capacity, D, scale, window, first,
                  softcap, sinks, workspace, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t tfa_kv4_prefill_workspace(int B, int Hq, int Hkv, int L, int S, int D, int window, int first) {
    if (B < 1 || Hkv < 1 || Hq < 1 || L < 1 || S < L || D < 1 || first < 0) return 0;
    const Seen sn = seen(L, S, window, first);
    return few_rows(B, Hq, Hkv, L, D, sn) ? decode_workspace(D) : static_cast<size_t>(B) * Hkv * sn.rows() * D * 4;
}

// The positions that are brought back, min(S, first + L + window - 1) with a window and
// S without, grow with L and S, and the other kernel's size is a constant.
extern "C" size_t tfa_kv4_prefill_workspace_most(int B, int Hq, int Hkv, int L, int S, int D, int window, int first) {
    if (B < 1 || Hkv < 1 || Hq < 1 || L < 1 || S < L || D < 1 || first < 0) return 0;
    const size_t dense = static_cast<size_t>(B) * Hkv * seen(L, S, window, first).rows() * D * 4, few = decode_workspace(D);
    return dense > few ? dense : few;
}

// A long chunk's products are the tensor core's to bound, so K and V are brought back
// to bf16 once (a rounding of each value, as a bf16 cache has), next to which they would
// be read by every query tile, and the dense kernel runs on them.  Only positions that
// some row sees are brought back; leaving the others out shifts rows and window alike.
extern "C" int tfa_kv4_prefill(const void *q, const void *k_codes, const void *k_meta, const void *v_codes,
                               const void *v_meta, void *o, int B, int Hq, int Hkv, int L, int S, int capacity, int D,
                               float scale, int window, int first, float softcap, const float *sinks, void *workspace,
                               tfa_stream_t stream) {
    if (!q || !o || !workspace) return TFA_ERR_NULL;
    if (int rc = check_cache(k_codes, k_meta, v_codes, v_meta, B, Hkv, capacity, D)) return rc;
    if (Hq < 1 || Hq % Hkv != 0) return TFA_ERR_HEADS;
    if (L < 1 || S < L || static_cast<long long>(B) * Hq * L > (1ll << 31) - 1) return TFA_ERR_SHAPE;
    if (S > capacity) return TFA_ERR_CACHE;
    if (first < 0 || (first > 0 && window <= 0)) return TFA_ERR_WINDOW;
    if (!std::isfinite(scale)) return TFA_ERR_SCALE;
    if (!std::isfinite(softcap) || softcap < 0.f || (softcap > 0.f && scale == 0.f)) return TFA_ERR_SOFTCAP;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(sinks, 4) || !aligned(workspace, 16)) return TFA_ERR_ALIGN;
    const Seen sn = seen(L, S, window, first);
    if (few_rows(B, Hq, Hkv, L, D, sn))
        return decode(q, k_codes, k_meta, v_codes, v_meta, nullptr, S, o, B, Hq, Hkv, L, capacity, D, scale, window, first,
                      softcap, sinks, workspace, reinterpret_cast<cudaStream_t>(stream));
    const int rows = static_cast<int>(sn.rows());
    const long long all = static_cast<long long>(B) * Hkv * rows;
    const unsigned blocks = row_blocks(all, D);
    if (all > (1ll << 31) - 1 || !blocks ||
        static_cast<long long>(B) * Hq * ((L + 255) / 256) > (1ll << 30))  // the dense kernel's own limits
        return TFA_ERR_SHAPE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ReadParams p = {};
    int sms = 0;
    if (int rc = tfa::device_info(s, &p.status, &sms)) return rc;
    p.c = cache_of(const_cast<void *>(k_codes), const_cast<void *>(k_meta), const_cast<void *>(v_codes),
                   const_cast<void *>(v_meta));
    p.k = static_cast<__nv_bfloat16 *>(workspace);
    p.v = p.k + static_cast<size_t>(all) * D;
    p.n_rows = static_cast<unsigned>(B) * Hkv * rows;
    p.Hkv = divisor(Hkv);
    p.rows = divisor(rows);
    p.cap = capacity;
    p.split = sn.lo > 0 ? sn.keep : rows;
    p.skip = sn.lo - sn.keep;
    if (int rc = launch_read(p, blocks, D, s)) return rc;
    if (window > 0 && first > 0)
        return tfa_prefill_first(q, p.k, p.v, o, nullptr, B, Hq, Hkv, L, rows, D, scale, window, first, nullptr, softcap,
                                 sinks, stream);
    return tfa_attention_ex(q, p.k, p.v, o, B, Hq, Hkv, L, rows, D, scale, 1, window, nullptr, softcap, sinks, stream);
}
