// cg_quant.cu -- tokens written into, and read back from, a paged pool held in
// 4 or 8 bits (sm_103a).
//
// A thread takes eight channels at a time: 16 bytes of the 16-bit tensor, 4
// or 8 of codes.  The 4, 8 or 16 threads of a group find its smallest and
// largest value by exchange, so that a row is read once and its codes go out
// in runs of 128 or 256 bytes a warp.
#include "cg_async.cuh"
#include "cg_quant.cuh"

namespace cg {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kKeep = 1024;  // sequences whose first rows a block keeps in shared memory

template <class T> struct Type;
template <> struct Type<__half> {
    using T2 = __half2;
    static __device__ __forceinline__ float2 wide(T2 x) { return __half22float2(x); }
    static __device__ __forceinline__ T2 pack(float a, float b) { return __floats2half2_rn(a, b); }
    static __device__ __forceinline__ T2 two(__half a, __half b) { return __halves2half2(a, b); }
    static __device__ __forceinline__ float of(uint32_t bits) { return __half2float(__ushort_as_half((uint16_t)bits)); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __half_as_ushort(__float2half_rn(x)); }
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

// A block takes a run of kU x 256 eight-channel units of the flattened rows,
// finds their tokens' places once, and then goes over `slices` layers of K and
// V, in which the places are the same.
struct Job {
    QuantPool p;
    TokenRows t;
    uint32_t *status;
    uint32_t units;            // of a row
    uint32_t runs;             // of a layer's K
    uint32_t slices, n_slices; // of a block; all of them: layers x 2
};

constexpr uint32_t kMaxRows = 4 * kThreads / 8 + 1;  // rows that a run touches: C is 64 at least

template <uint32_t kU> struct Run {
    uint64_t at[kU];    // word offset of the row in a layer's K, or kNone / kOutside
    uint32_t row[kU], unit[kU];
    uint32_t slice, end;
    __device__ __forceinline__ Run(const Job &b) {
        __shared__ uint32_t sh_first[kKeep + 1];
        __shared__ uint64_t sh_at[kMaxRows];
        const uint32_t *first = b.t.first;
        if (first && b.t.n_seqs <= kKeep) {
            for (uint32_t k = threadIdx.x; k <= b.t.n_seqs; k += kThreads) sh_first[k] = first[k];
            first = sh_first;
            __syncthreads();
        }
        const uint32_t part = blockIdx.x / b.runs, run = blockIdx.x - part * b.runs;
        const uint64_t from = (uint64_t)run * (kU * kThreads);
        const uint32_t j0 = from >> 32 ? (uint32_t)(from / b.units) : (uint32_t)from / b.units;
        const uint32_t x0 = (uint32_t)(from - (uint64_t)j0 * b.units), rows = (x0 + kU * kThreads - 1) / b.units + 1;
        for (uint32_t k = threadIdx.x; k < rows; k += kThreads)
            sh_at[k] = j0 + k < b.t.n_rows ? place(b.p, b.t, first, j0 + k, b.status) : kNone;
        __syncthreads();
#pragma unroll
        for (uint32_t u = 0; u < kU; u++) {
            const uint32_t x = x0 + u * kThreads + threadIdx.x, k = x / b.units;
            row[u] = j0 + k;
            unit[u] = x - k * b.units;
            at[u] = sh_at[k];
        }
        slice = part * b.slices;
        end = min(slice + b.slices, b.n_slices);
    }
};

template <class T, uint32_t kBits, uint32_t kU>
__global__ void __launch_bounds__(kThreads) k_quant_write(const Job b) {
    using Y = Type<T>;
    constexpr float kTop = (1u << kBits) - 1u, kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer
    const Run<kU> r(b);
    const uint32_t lanes = b.p.group / 8;
    for (uint32_t slice = r.slice; slice < r.end; slice++) {
        const uint32_t layer = slice >> 1, kv = slice & 1u;
        const uint16_t *src = kv ? b.t.v + layer * b.t.vs[0] : b.t.k + layer * b.t.ks[0];
        const uint64_t stride = kv ? b.t.vs[1] : b.t.ks[1];
        uint16_t *pool = b.p.pool + layer * b.p.layer + kv * b.p.kv;
        uint4 in[kU];
#pragma unroll
        for (uint32_t u = 0; u < kU; u++)
            in[u] = r.at[u] < kOutside ? *reinterpret_cast<const uint4 *>(src + r.row[u] * stride + 8 * r.unit[u]) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (uint32_t u = 0; u < kU; u++) {
            const typename Y::T2 *h = reinterpret_cast<const typename Y::T2 *>(&in[u]);
            typename Y::T2 mn = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
            typename Y::T2 mx = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
            // both in one word: the larger of x and -x's
            typename Y::T2 mm = Y::two(__hmax_nan(mx.x, mx.y), __hneg(__hmin_nan(mn.x, mn.y)));
            mm = __hmax2_nan(mm, __shfl_xor_sync(kFull, mm, 1));
            mm = __hmax2_nan(mm, __shfl_xor_sync(kFull, mm, 2));
            if (lanes > 4) mm = __hmax2_nan(mm, __shfl_xor_sync(kFull, mm, 4));
            if (lanes > 8) mm = __hmax2_nan(mm, __shfl_xor_sync(kFull, mm, 8));
            if (r.at[u] >= kOutside) continue;
            const float2 hl = Y::wide(mm);
            const float low = -hl.y, d = hl.x - low;
            const bool finite = d - d == 0.f;
            // the smallest scale of the type with scale * kTop >= d: the products are exact, the first guess is at
            // most one step off
            uint32_t sb = Y::bits(d * (1.f / kTop));
            if (sb && Y::of(sb - 1) * kTop >= d) sb--;
            if (Y::of(sb) * kTop < d) sb++;
            const float s = Y::of(sb);
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
            if (!sb) inv = 0.f;
            // codes: the nearest integers to (x - low) / s, unless one is near a border (or 1 / s too large)
            float y[8], c[8], far = s < 0x1p-90f && sb ? 1.f : 0.f;
#pragma unroll
            for (uint32_t k = 0; k < 4; k++) {
                const float2 x = Y::wide(h[k]);
                float q[2], e[2];
                y[2 * k] = x.x, y[2 * k + 1] = x.y;
                add2(y[2 * k], y[2 * k + 1], -low, -low);
                fma2(q[0], q[1], y[2 * k], y[2 * k + 1], inv, kMagic);
                c[2 * k] = q[0], c[2 * k + 1] = q[1];
                add2(c[2 * k], c[2 * k + 1], -kMagic, -kMagic);
                e[0] = fmaf(y[2 * k], inv, -c[2 * k]), e[1] = fmaf(y[2 * k + 1], inv, -c[2 * k + 1]);
                far = fmaxf(far, fmaxf(fabsf(e[0]), fabsf(e[1])));
            }
            if (far > 0.4995f && finite)
#pragma unroll
                for (uint32_t k = 0; k < 8; k++)
                    if (far >= 1.f || fabsf(fmaf(y[k], inv, -c[k])) > 0.4995f) c[k] = code_at_border(y[k], s);
            uint16_t *row = pool + r.at[u];
            if constexpr (kBits == 4) {
                uint32_t w[2];
#pragma unroll
                for (uint32_t k = 0; k < 2; k++)
                    w[k] = __float_as_uint(fmaf(c[4 * k + 3], 4096.f, fmaf(c[4 * k + 2], 256.f, fmaf(c[4 * k + 1], 16.f, c[4 * k]))) + 8388608.f);
                reinterpret_cast<uint32_t *>(row)[r.unit[u]] = finite ? __byte_perm(w[0], w[1], 0x5410) : 0u;
            } else {
                uint32_t w[2];
#pragma unroll
                for (uint32_t k = 0; k < 2; k++)
                    w[k] = __byte_perm(__float_as_uint(fmaf(c[4 * k + 1], 256.f, c[4 * k]) + 8388608.f),
                                       __float_as_uint(fmaf(c[4 * k + 3], 256.f, c[4 * k + 2]) + 8388608.f), 0x5410);
                reinterpret_cast<uint2 *>(row)[r.unit[u]] = finite ? make_uint2(w[0], w[1]) : make_uint2(0, 0);
            }
            if ((threadIdx.x & (lanes - 1)) == 0) {
                reinterpret_cast<uint32_t *>(row + b.p.codes)[r.unit[u] / lanes] = finite ? sb | Y::bits(low) << 16 : Y::kNan << 16;
                if (!finite) flag(b.status, CG_ERR_NONFINITE);
            }
        }
    }
}

template <class T, uint32_t kBits, uint32_t kU>
__global__ void __launch_bounds__(kThreads) k_quant_read(const Job b) {
    using Y = Type<T>;
    const Run<kU> r(b);
    const uint32_t glog = 31 - __clz(b.p.group / 8);
    for (uint32_t slice = r.slice; slice < r.end; slice++) {
        const uint32_t layer = slice >> 1, kv = slice & 1u;
        uint16_t *dst = kv ? b.t.v + layer * b.t.vs[0] : b.t.k + layer * b.t.ks[0];
        const uint64_t stride = kv ? b.t.vs[1] : b.t.ks[1];
        const uint16_t *pool = b.p.pool + layer * b.p.layer + kv * b.p.kv;
        uint2 w[kU];
        uint32_t pair[kU];
#pragma unroll
        for (uint32_t u = 0; u < kU; u++) {
            w[u] = make_uint2(0, 0);
            pair[u] = 0;
            if (r.at[u] < kOutside) {
                const uint16_t *row = pool + r.at[u];
                if constexpr (kBits == 4) w[u].x = reinterpret_cast<const uint32_t *>(row)[r.unit[u]];
                else w[u] = reinterpret_cast<const uint2 *>(row)[r.unit[u]];
                pair[u] = reinterpret_cast<const uint32_t *>(row + b.p.codes)[r.unit[u] >> glog];
            }
        }
#pragma unroll
        for (uint32_t u = 0; u < kU; u++) {
            if (r.at[u] >= kOutside && !(r.at[u] == kOutside && b.t.zero)) continue;
            const float s = Y::of(pair[u] & 0xFFFFu), low = Y::of(pair[u] >> 16);
            float x[8], most = -INFINITY;
#pragma unroll
            for (uint32_t k = 0; k < 8; k += 2) {
                uint32_t c[2];
#pragma unroll
                for (uint32_t e = 0; e < 2; e++) {  // 2^23 + code
                    if constexpr (kBits == 4) c[e] = ((w[u].x >> (4 * (k + e))) & 15u) | 0x4B000000u;
                    else c[e] = __byte_perm(k < 4 ? w[u].x : w[u].y, 0x4B000000u, 0x7440u | ((k + e) & 3u));
                    x[k + e] = __uint_as_float(c[e]);
                }
                add2(x[k], x[k + 1], -8388608.f, -8388608.f);
                x[k] = fmaf(x[k], s, low), x[k + 1] = fmaf(x[k + 1], s, low);
                most = fmaxf(most, fmaxf(x[k], x[k + 1]));
            }
            if (most > Y::kMost)  // past the type's range
#pragma unroll
                for (uint32_t k = 0; k < 8; k++) x[k] = x[k] > Y::kMost && x[k] < INFINITY ? Y::kMost : x[k];
            uint4 o;
            typename Y::T2 *h = reinterpret_cast<typename Y::T2 *>(&o);
#pragma unroll
            for (uint32_t k = 0; k < 4; k++) h[k] = Y::pack(x[2 * k], x[2 * k + 1]);
            const uint64_t at = r.row[u] * stride + 8 * r.unit[u];
            *reinterpret_cast<uint4 *>(dst + at) = o;
            if (b.t.k_rest && !kv) {
#pragma unroll
                for (uint32_t k = 0; k < 4; k++) {
                    const float2 y = Y::wide(h[k]);
                    h[k] = Y::pack(x[2 * k] - y.x, x[2 * k + 1] - y.y);
                }
                *reinterpret_cast<uint4 *>(b.t.k_rest + at) = o;
            }
        }
    }
}

template <class T, uint32_t kBits>
cudaError_t launch(Job &b, uint32_t n_layers, bool write, cudaStream_t s) {
    b.units = b.p.C / 8;
    b.n_slices = 2 * n_layers;
    const uint64_t n = (uint64_t)b.t.n_rows * b.units;  // of a layer's K
    // one unit a thread where the call is short, four where that leaves every SM full; and eight slices a block
    const bool wide = n * b.n_slices >= 4ull * 152 * 2048;
    const uint64_t per = (wide ? 4u : 1u) * kThreads, runs = (n + per - 1) / per, full = 152 * 8;
    b.slices = 8;
    while (b.slices > 1 && runs * ((b.n_slices + b.slices - 1) / b.slices) < 4 * full) b.slices >>= 1;
    const uint64_t grid = runs * ((b.n_slices + b.slices - 1) / b.slices);
    if (grid > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    b.runs = (uint32_t)runs;
    if (write) {
        if (wide) k_quant_write<T, kBits, 4><<<(unsigned)grid, kThreads, 0, s>>>(b);
        else k_quant_write<T, kBits, 1><<<(unsigned)grid, kThreads, 0, s>>>(b);
    } else {
        if (wide) k_quant_read<T, kBits, 4><<<(unsigned)grid, kThreads, 0, s>>>(b);
        else k_quant_read<T, kBits, 1><<<(unsigned)grid, kThreads, 0, s>>>(b);
    }
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
    // blocks of at least 256 eight-channel units: the grid must fit
    if ((uint64_t)r->n_rows * (quant_channels(f) / 8) / kThreads * 2 * r->n_layers > 0x7FFF0000ull) return CG_ERR_INVALID_ARG;
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
