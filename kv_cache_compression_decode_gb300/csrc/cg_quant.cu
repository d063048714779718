// cg_quant.cu -- tokens written into, and read back from, a paged pool held in
// 4 or 8 bits (sm_103a).
//
// A lane takes eight channels at a time: 16 bytes of the 16-bit tensor, 4 or 8
// of codes.  The 4, 8 or 16 lanes of a group find its smallest and largest
// value by exchange, so that a row is read once and its codes go out in runs of
// 128 or 256 bytes a warp.
#include "cg_async.cuh"
#include "cg_launch.cuh"
#include "cg_quant.cuh"

namespace cg {
namespace {

constexpr uint32_t kThreads = 256;

template <class T> struct Type;
template <> struct Type<__half> {
    using T2 = __half2;
    static __device__ __forceinline__ float2 wide(T2 x) { return __half22float2(x); }
    static __device__ __forceinline__ T2 pack(float a, float b) { return __floats2half2_rn(a, b); }
    static __device__ __forceinline__ T2 two(__half a, __half b) { return __halves2half2(a, b); }
    static __device__ __forceinline__ float of(uint32_t bits) { return __half2float(__ushort_as_half((uint16_t)bits)); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __half_as_ushort(__float2half_rn(x)); }
    static __device__ __forceinline__ uint32_t bits_up(float x) { return __half_as_ushort(__float2half_ru(x)); }
    // the two of a word plus z, in fp32
    static __device__ __forceinline__ void add(float &x, float &y, uint32_t w, float z) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.rn.f32.f16 %0, a, %3;\n\tadd.rn.f32.f16 %1, b, %3;\n\t}"
            : "=f"(x), "=f"(y)
            : "r"(w), "f"(z));
    }
    static constexpr uint32_t kNan = 0x7E00u;
    static constexpr float kMost = 65504.f;
};
template <> struct Type<__nv_bfloat16> {
    using T2 = __nv_bfloat162;
    static __device__ __forceinline__ float2 wide(T2 x) { return __bfloat1622float2(x); }
    static __device__ __forceinline__ T2 pack(float a, float b) { return __floats2bfloat162_rn(a, b); }
    static __device__ __forceinline__ T2 two(__nv_bfloat16 a, __nv_bfloat16 b) { return __halves2bfloat162(a, b); }
    static __device__ __forceinline__ float of(uint32_t bits) { return __uint_as_float(bits << 16); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
    static __device__ __forceinline__ uint32_t bits_up(float x) { return (__float_as_uint(x) + 0xFFFFu) >> 16; }  // x >= 0
    // the two of a word plus z, in fp32
    static __device__ __forceinline__ void add(float &x, float &y, uint32_t w, float z) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.rn.f32.bf16 %0, a, %3;\n\tadd.rn.f32.bf16 %1, b, %3;\n\t}"
            : "=f"(x), "=f"(y)
            : "r"(w), "f"(z));
    }
    static constexpr uint32_t kNan = 0x7FC0u;
    static constexpr float kMost = 3.3895313892515355e38f;  // (2 - 2^-7) 2^127
};

// The sequence that row j belongs to (n_seqs: none): the last r with first[r] <= j, if j < first[r + 1].
__device__ __forceinline__ uint32_t owner(const TokenRows &t, const uint32_t *first, uint32_t j, uint32_t &at, uint32_t &count) {
    if (!t.first) {
        const uint32_t r = j / t.per;
        at = j - r * t.per;
        count = t.per;
        return r;
    }
    uint32_t lo = 0, hi = t.n_seqs;  // first[hi] > j, or hi is the end
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (first[mid] <= j) lo = mid;
        else hi = mid;
    }
    const uint32_t f0 = first[lo], f1 = first[lo + 1];
    at = j - f0;
    count = f1 - f0;
    return j >= f0 && j < f1 ? lo : t.n_seqs;
}

// Where row j's token lies: word offset within a layer's K.  kNone: the row is
// not used; kOutside: its block is not in the pool.
constexpr uint64_t kNone = ~0ull, kOutside = ~0ull - 1;
__device__ __forceinline__ uint64_t place(const QuantPool &p, const TokenRows &t, const uint32_t *first, uint32_t j,
                                          uint32_t *status) {
    uint32_t at, count;
    const uint32_t r = owner(t, first, j, at, count);
    if (r >= t.n_seqs) return kNone;
    const uint32_t s = t.slots ? t.slots[r] : t.slot0 + r;
    if (s >= p.n_slots) {
        flag(status, CG_ERR_RANGE);
        return kNone;
    }
    const uint32_t n = t.fixed ? t.fixed : p.lens[s];
    if (n == 0) return kNone;
    const uint64_t begin = t.start ? t.start[r] : (uint64_t)n - count;
    if ((!t.start && count > n) || (t.start && begin + count > n) || n > ((uint64_t)p.n_blocks << p.bshift)) {
        flag(status, CG_ERR_RANGE);
        return kNone;
    }
    const uint32_t pos = (uint32_t)begin + at, id = p.tables[(uint64_t)s * p.n_blocks + (pos >> p.bshift)];
    if (id >= p.n_pool) {
        flag(status, CG_ERR_RANGE);
        return kOutside;
    }
    return id * p.block + (pos & ((1u << p.bshift) - 1u)) * p.token;
}

// The code of y = x - low where y / s lies near a border between two codes or
// s is very small: decided by the sign of y - (n + 1/2) s, whose product is
// exact in fp32 (a 9-bit number times an 11-bit one).
__device__ __noinline__ float code_at_border(float y, float s) {
    const float n = floorf(__fdiv_rn(y, s)), h = (n + 0.5f) * s;
    if (y != h) return y > h ? n + 1.f : n;
    return n + ((int)n & 1);
}

// A warp, or an eighth to a half of one where rows are short, takes a row: its
// lanes find the token's place and go over the row's eight-channel units side
// by side, kBatch of them in flight, in K and V of some layers, in which the
// place is the same.
constexpr uint32_t kBatch = 4;
struct Job {
    QuantPool p;
    TokenRows t;
    uint32_t *status;
    uint32_t llog;             // log2 of the lanes of a row
    uint32_t units;            // of a row
    uint32_t steps, chunks;    // steps of a warp along a row; how many warps share a row
    uint32_t slices, n_slices; // of a warp; all of them: layers x (K, V)
};

struct Run {
    uint32_t j, unit, end;  // row; this lane's first unit, end of the warp's units
    uint64_t at;            // place, or kNone / kOutside
    uint32_t slice, last;
    bool some;              // some lane of the warp has a row
    __device__ __forceinline__ Run(const Job &b) {
        const uint32_t lane = threadIdx.x & 31u, id = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
        const uint32_t group = b.chunks == 1 ? id : id / b.chunks, chunk = b.chunks == 1 ? 0u : id - group * b.chunks;
        const uint64_t row = ((uint64_t)group << (5u - b.llog)) + (lane >> b.llog);
        j = (uint32_t)row;
        unit = ((chunk * b.steps) << b.llog) + (lane & ((1u << b.llog) - 1u));
        end = min(b.units, ((chunk + 1u) * b.steps) << b.llog);
        at = row < b.t.n_rows ? place(b.p, b.t, b.t.first, j, b.status) : kNone;
        slice = blockIdx.y * b.slices;
        last = min(slice + b.slices, b.n_slices);
        some = __any_sync(kFull, at != kNone);
    }
};

// Codes and pair of a unit; its group's `lanes` threads call together.
template <class T, uint32_t kBits>
__device__ __forceinline__ bool quantise(const uint4 &in, uint32_t lanes, uint2 &codes, uint32_t &pair) {
    using Y = Type<T>;
    constexpr float kTop = (1u << kBits) - 1u, kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer
    const typename Y::T2 *h = reinterpret_cast<const typename Y::T2 *>(&in);
    typename Y::T2 mn = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
    typename Y::T2 mx = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    // both in one word: the larger of x and -x's
    typename Y::T2 mm = Y::two(__hmax_nan(mx.x, mx.y), __hneg(__hmin_nan(mn.x, mn.y)));
    mm = __hmax2_nan(mm, __shfl_xor_sync(kFull, mm, 1));
    mm = __hmax2_nan(mm, __shfl_xor_sync(kFull, mm, 2));
    if (lanes > 4) mm = __hmax2_nan(mm, __shfl_xor_sync(kFull, mm, 4));
    if (lanes > 8) mm = __hmax2_nan(mm, __shfl_xor_sync(kFull, mm, 8));
    const float2 hl = Y::wide(mm);
    const float low = -hl.y, d = hl.x - low;
    // The smallest scale of the type with scale * kTop >= d.  d (1 - 2^-21) / kTop, rounded up to the type, is that or
    // the number before it; the products are exact.
    uint32_t sb = Y::bits_up(d * ((1.f - 0x1p-21f) / kTop));
    if (Y::of(sb) * kTop < d) sb++;
    const float s = Y::of(sb);
    float inv;  // of 2^-126 at least: with a scale of 0 every x - low is 0, too
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaxf(s, 0x1p-126f)));
    // Codes are the nearest integers to (x - low) / s.  The quotients are off by 2^-22 of themselves at most: a code
    // that is not near a border is right (and with bf16's smallest scales, whose inverse is not, none is trusted).
    float y[8], c[8], far = 0.f;
    if constexpr (!__is_same(T, __half)) far = sb && s < 0x1p-90f ? 1.f : 0.f;
    const uint32_t words[4] = {in.x, in.y, in.z, in.w};
    constexpr float kNear = 0.5f - kTop * 0x1p-20f;
#pragma unroll
    for (uint32_t k = 0; k < 4; k++) {
        Y::add(y[2 * k], y[2 * k + 1], words[k], -low);
        fma2(c[2 * k], c[2 * k + 1], y[2 * k], y[2 * k + 1], inv, kMagic);
        add2(c[2 * k], c[2 * k + 1], -kMagic, -kMagic);
        far = fmaxf(far, fmaxf(fabsf(fmaf(y[2 * k], inv, -c[2 * k])), fabsf(fmaf(y[2 * k + 1], inv, -c[2 * k + 1]))));
    }
    const bool finite = d - d == 0.f;
    if (far > kNear && finite)
#pragma unroll
        for (uint32_t k = 0; k < 8; k++)
            if (far >= 1.f || fabsf(fmaf(y[k], inv, -c[k])) > kNear) c[k] = code_at_border(y[k], s);
    // codes side by side, as integers
    uint32_t w[2];
    if constexpr (kBits == 4) {
#pragma unroll
        for (uint32_t k = 0; k < 2; k++)
            w[k] = __float_as_uint(fmaf(c[4 * k + 3], 4096.f, fmaf(c[4 * k + 2], 256.f, fmaf(c[4 * k + 1], 16.f, c[4 * k]))) + 8388608.f);
        codes.x = __byte_perm(w[0], w[1], 0x5410);
    } else {
#pragma unroll
        for (uint32_t k = 0; k < 2; k++)
            w[k] = __byte_perm(__float_as_uint(fmaf(c[4 * k + 1], 256.f, c[4 * k]) + 8388608.f),
                               __float_as_uint(fmaf(c[4 * k + 3], 256.f, c[4 * k + 2]) + 8388608.f), 0x5410);
        codes = make_uint2(w[0], w[1]);
    }
    // low as it came: mm holds -low above the largest value
    const uint32_t both = *reinterpret_cast<const uint32_t *>(&mm);
    pair = __byte_perm(sb, both ^ 0x80000000u, 0x7610);
    if (!finite) {
        codes = make_uint2(0, 0);
        pair = Y::kNan << 16;
    }
    return finite;
}

// Bound by the issue of instructions, 130 for a warp's 32 units, of which the
// codes are 65 (75% of the cycles issue one): 9001 tokens x 32 layers x 1024
// channels in 4 bits take 343 us, 4.55 TB/s.  Four blocks an SM (64 registers)
// beat three and five: 588 / 606 / 602 us with the read after it.
template <class T, uint32_t kBits>
__global__ void __launch_bounds__(kThreads, 4) k_quant_write(const Job b) {
    const Run r(b);
    if (!r.some) return;
    const uint32_t lanes = b.p.group / 8, glog = 31u - __clz(lanes), step = 1u << b.llog;
    const bool here = r.at < kOutside, first = here && (threadIdx.x & (lanes - 1u)) == 0;
    for (uint32_t slice = r.slice; slice < r.last; slice++) {
        const uint32_t layer = slice >> 1, kv = slice & 1u;
        const uint16_t *src = kv ? b.t.v + layer * b.t.vs[0] + r.j * b.t.vs[1] : b.t.k + layer * b.t.ks[0] + r.j * b.t.ks[1];
        uint32_t *row = reinterpret_cast<uint32_t *>(b.p.pool + layer * b.p.layer + kv * b.p.kv + (here ? r.at : 0));
        uint32_t *pairs = row + b.p.codes / 2;
        for (uint32_t u0 = r.unit; __any_sync(kFull, u0 < r.end); u0 += kBatch * step) {
            uint4 in[kBatch];
#pragma unroll
            for (uint32_t u = 0; u < kBatch; u++) {
                const uint32_t unit = u0 + u * step;
                in[u] = here && unit < r.end ? *reinterpret_cast<const uint4 *>(src + 8 * unit) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (uint32_t u = 0; u < kBatch; u++) {
                const uint32_t unit = u0 + u * step;
                if (u && !__any_sync(kFull, unit < r.end)) break;
                uint2 codes;
                uint32_t pair;
                const bool finite = quantise<T, kBits>(in[u], lanes, codes, pair);
                if (!here || unit >= r.end) continue;
                if constexpr (kBits == 4) row[unit] = codes.x;
                else reinterpret_cast<uint2 *>(row)[unit] = codes;
                if (first) pairs[unit >> glog] = pair;
                if (!finite) flag(b.status, CG_ERR_NONFINITE);
            }
        }
    }
}

// Bound by DRAM: 15000 tokens x 32 layers in 8 bits take 441 us, 6.63 TB/s, 98%
// of a plain copy's rate; in 4 bits instructions count, 9001 x 32 take 245 us,
// 6.05 TB/s.  (A block that found its rows' places together, a thread at a time
// going over their units, took 478 and 282 us: a warp to a row needs no barrier
// and one address for all of it.)
template <class T, uint32_t kBits>
__global__ void __launch_bounds__(kThreads) k_quant_read(const Job b) {
    using Y = Type<T>;
    constexpr float kTop = (1u << kBits) - 1u;
    let_next_start();
    const Run r(b);
    const bool here = r.at < kOutside, use = here || (b.t.zero && r.at == kOutside);
    if (!use) return;
    const uint32_t glog = 31u - __clz(b.p.group / 8), step = 1u << b.llog;
    for (uint32_t slice = r.slice; slice < r.last; slice++) {
        const uint32_t layer = slice >> 1, kv = slice & 1u;
        uint16_t *dst = kv ? b.t.v + layer * b.t.vs[0] + r.j * b.t.vs[1] : b.t.k + layer * b.t.ks[0] + r.j * b.t.ks[1];
        uint16_t *rest = !kv && b.t.k_rest ? b.t.k_rest + (dst - b.t.k) : nullptr;
        const uint32_t *row = reinterpret_cast<const uint32_t *>(b.p.pool + layer * b.p.layer + kv * b.p.kv + (here ? r.at : 0));
        const uint32_t *pairs = row + b.p.codes / 2;
        for (uint32_t u0 = r.unit; u0 < r.end; u0 += kBatch * step) {
            uint2 w[kBatch];
            uint32_t pair[kBatch];
#pragma unroll
            for (uint32_t u = 0; u < kBatch; u++) {
                const uint32_t unit = u0 + u * step;
                w[u] = make_uint2(0, 0);
                pair[u] = 0;
                if (here && unit < r.end) {
                    if constexpr (kBits == 4) w[u].x = row[unit];
                    else w[u] = reinterpret_cast<const uint2 *>(row)[unit];
                    pair[u] = pairs[unit >> glog];
                }
            }
#pragma unroll
            for (uint32_t u = 0; u < kBatch; u++) {
                const uint32_t unit = u0 + u * step;
                if (unit >= r.end) break;
                const float s = Y::of(pair[u] & 0xFFFFu), low = Y::of(pair[u] >> 16);
                float x[8];
                if constexpr (kBits == 4) {
                    // codes k and k + 4 in place: 2^23 + code 16^k, less 2^23, times s / 16^k
                    const uint32_t y[2] = {w[u].x, w[u].x >> 16};
                    float f = s;
#pragma unroll
                    for (uint32_t k = 0; k < 4; k++) {
                        x[k] = __uint_as_float((y[0] & (15u << 4 * k)) | 0x4B000000u);
                        x[k + 4] = __uint_as_float((y[1] & (15u << 4 * k)) | 0x4B000000u);
                        add2(x[k], x[k + 4], -8388608.f, -8388608.f);
                        fma2(x[k], x[k + 4], x[k], x[k + 4], f, low);
                        f *= 0.0625f;
                    }
                } else {
#pragma unroll
                    for (uint32_t k = 0; k < 8; k += 2) {
#pragma unroll
                        for (uint32_t e = 0; e < 2; e++)
                            x[k + e] = __uint_as_float(__byte_perm(k < 4 ? w[u].x : w[u].y, 0x4B000000u, 0x7440u | ((k + e) & 3u)));
                        add2(x[k], x[k + 1], -8388608.f, -8388608.f);
                        fma2(x[k], x[k + 1], x[k], x[k + 1], s, low);
                    }
                }
                if (fmaf(kTop, s, low) > Y::kMost) {  // some may lie past the type's range (bf16's past fp32's, too)
                    const float most = s < INFINITY && low < INFINITY ? Y::kMost : INFINITY;
#pragma unroll
                    for (uint32_t k = 0; k < 8; k++) x[k] = x[k] > Y::kMost ? most : x[k];
                }
                uint4 o;
                typename Y::T2 *h = reinterpret_cast<typename Y::T2 *>(&o);
#pragma unroll
                for (uint32_t k = 0; k < 4; k++) h[k] = Y::pack(x[2 * k], x[2 * k + 1]);
                *reinterpret_cast<uint4 *>(dst + 8 * unit) = o;
                if (rest) {
#pragma unroll
                    for (uint32_t k = 0; k < 4; k++) {
                        const float2 y = Y::wide(h[k]);
                        h[k] = Y::pack(x[2 * k] - y.x, x[2 * k + 1] - y.y);
                    }
                    *reinterpret_cast<uint4 *>(rest + 8 * unit) = o;
                }
            }
        }
    }
}

// Where the call is short, a warp takes 32 units of K or of V of one layer;
// otherwise whole rows, in up to eight layers as long as there are warps
// enough.
template <class T, uint32_t kBits>
cudaError_t launch(Job &b, uint32_t n_layers, bool write, cudaStream_t s) {
    b.units = b.p.C / 8;
    b.n_slices = 2 * n_layers;
    b.llog = b.units >= 32 ? 5 : b.units >= 16 ? 4 : 3;
    const uint64_t groups = ((uint64_t)b.t.n_rows + (32u >> b.llog) - 1) >> (5 - b.llog);
    const uint32_t steps = (b.units + (1u << b.llog) - 1) >> b.llog;
    const uint64_t full = 152 * 32;  // warps that fill the SMs
    b.steps = steps;
    b.slices = 16;
    const auto warps = [&] { return groups * ((steps + b.steps - 1) / b.steps) * ((b.n_slices + b.slices - 1) / b.slices); };
    while (b.slices > 2 && warps() < 2 * full) b.slices >>= 1;
    if (warps() < full) b.slices = 1;
    while (b.steps > 1 && warps() < full) b.steps = (b.steps + 1) / 2;
    while ((b.n_slices + b.slices - 1) / b.slices > 65535u) b.slices <<= 1;
    b.chunks = (steps + b.steps - 1) / b.steps;
    const uint64_t runs = (groups * b.chunks + kThreads / 32 - 1) / (kThreads / 32);
    if (runs > 0x7FFFFFFFull / (kThreads / 32)) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)runs, (b.n_slices + b.slices - 1) / b.slices);
    if (write) k_quant_write<T, kBits><<<grid, kThreads, 0, s>>>(b);
    else k_quant_read<T, kBits><<<grid, kThreads, 0, s>>>(b);
    return cudaGetLastError();
}

cudaError_t run(const QuantPool &p, const TokenRows &t, uint32_t n_layers, uint32_t dtype, uint32_t bits, bool write,
                uint32_t *status, cudaStream_t s) {
    Job b{};
    b.p = p;
    b.t = t;
    b.status = status;
    if (dtype == CG_FP16) return bits == 4 ? launch<__half, 4>(b, n_layers, write, s) : launch<__half, 8>(b, n_layers, write, s);
    return bits == 4 ? launch<__nv_bfloat16, 4>(b, n_layers, write, s) : launch<__nv_bfloat16, 8>(b, n_layers, write, s);
}

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) != 0; }

cg_status tokens(const cg_pages *p, const cg_quant *f, const cg_token_rows *r, bool write, uint32_t *dev_status, void *stream) {
    if (!p || !r || !quant_ok(f) || !p->pool || !p->tables || !p->lens) return CG_ERR_INVALID_ARG;
    if (!p->L || !p->n_pool_blocks || !p->n_slots || !p->n_blocks || p->C != quant_row(f) || p->token_stride < p->C)
        return CG_ERR_INVALID_ARG;
    const uint32_t bt = p->block_tokens;
    if (!bt || (bt & (bt - 1u)) || (uint64_t)p->n_blocks * bt > (1ull << 31)) return CG_ERR_INVALID_ARG;
    if (r->layer >= p->L || r->n_layers > p->L - r->layer || !r->n_layers) return CG_ERR_INVALID_ARG;
    if (r->n_seqs > (1u << 31) || r->n_rows > (1u << 31)) return CG_ERR_INVALID_ARG;
    if (r->n_seqs == 0 || r->n_rows == 0) return CG_OK;
    if (!r->k || !r->v || (!r->first && r->n_rows % r->n_seqs)) return CG_ERR_INVALID_ARG;
    const auto used = [](uint64_t n, uint64_t stride) { return n > 1 ? stride : 0; };
    const uint64_t strides = used(p->L, p->layer_stride) | p->kv_stride | used(p->n_pool_blocks, p->block_stride) |
                             used(bt, p->token_stride) | used(r->n_layers, r->k_stride[0] | r->v_stride[0]) |
                             used(r->n_rows, r->k_stride[1] | r->v_stride[1]);
    if (strides % 8 || misaligned(p->pool, 16) || misaligned(r->k, 16) || misaligned(r->v, 16)) return CG_ERR_INVALID_ARG;
    if (misaligned(p->tables, 4) || misaligned(p->lens, 4) || misaligned(r->slots, 4) || misaligned(r->first, 4) ||
        misaligned(r->start, 4))
        return CG_ERR_INVALID_ARG;
    TokenRows t{};
    t.k = r->k;
    t.v = r->v;
    t.slots = r->slots;
    t.first = r->first;
    t.start = r->start;
    t.n_seqs = r->n_seqs;
    t.n_rows = r->n_rows;
    t.per = r->n_rows / r->n_seqs;
    for (int k = 0; k < 2; k++) {
        t.ks[k] = r->k_stride[k];
        t.vs[k] = r->v_stride[k];
    }
    // the number of warps must fit: one takes 32 eight-channel units of a row at least
    if ((uint64_t)r->n_rows * ((quant_channels(f) / 8 + 31) / 32) > 0x7FFF0000ull) return CG_ERR_INVALID_ARG;
    CG_CUDA_TRY(run(quant_pool(p, f, r->layer), t, r->n_layers, f->dtype, f->bits, write, dev_status,
                    static_cast<cudaStream_t>(stream)));
    return CG_OK;
}

}  // namespace

QuantPool quant_pool(const cg_pages *p, const cg_quant *f, uint32_t layer) {
    return QuantPool{p->pool + layer * p->layer_stride, p->tables, p->lens, p->n_slots, p->n_blocks, p->n_pool_blocks,
                     (uint32_t)__builtin_ctz(p->block_tokens), p->layer_stride, p->kv_stride, p->block_stride,
                     p->token_stride, quant_channels(f), quant_codes(f), f->group};
}

cudaError_t quant_read(const QuantPool &p, const TokenRows &rows, uint32_t n_layers, uint32_t dtype, uint32_t bits,
                       uint32_t *status, cudaStream_t s) {
    return run(p, rows, n_layers, dtype, bits, false, status, s);
}

}  // namespace cg

using namespace cg;

extern "C" cg_status cg_quant_row(const cg_quant *f, uint32_t *row) {
    if (!quant_ok(f) || !row) return CG_ERR_INVALID_ARG;
    *row = quant_row(f);
    return CG_OK;
}

extern "C" cg_status cg_quant_write(const cg_pages *p, const cg_quant *f, const cg_token_rows *rows,
                                    uint32_t *dev_status, void *stream) {
    return tokens(p, f, rows, true, dev_status, stream);
}

extern "C" cg_status cg_quant_read(const cg_pages *p, const cg_quant *f, const cg_token_rows *rows,
                                   uint32_t *dev_status, void *stream) {
    return tokens(p, f, rows, false, dev_status, stream);
}
