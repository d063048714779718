// cg_quant_rows.cuh -- query rows against the tokens of a pool in 4 or 8 bits
// (sm_103a).  Compiled once for each width of code and size of head
// (cg_quant_rows_*.cu).
//
// With value = low + code * scale for a group of channels,
//     <q, K_t>      = sum_g scale_tg <q_g, code_tg> + low_tg sum(q_g)
//     sum_t p_t V_t = sum_t (p_t scale_tg) code_tg + sum_t p_t low_tg
// so the matrix instructions take codes as they are: an integer below 2^8 in
// the low bits of an fp16 word is the denormal number code * 2^-24, which they
// multiply exactly, and a code becomes an operand by one AND (a 4-bit code four
// places higher is code * 2^-20: the other operand, or the result, carries the
// 2^-4).  Scales are applied in fp32.  The low values' part of the scores is one
// more product, of a token's pairs as they lie with the sums of q in parts.
//
// Codes are the larger operand's 16 rows (m16n8k16: a token's codes along the
// rows' contraction for the scores, a channel's along tokens for the output),
// query rows its 8 columns: the eight query heads of a KV head fill them, and a
// single one wastes no codes.  A warp's tokens are permuted (pi) so that its
// loads from the swizzled tiles meet no bank twice.  tcgen05 has no place here:
// its operands would have to be written to shared memory as 16-bit numbers
// first, which takes more instructions than the products do.
//
// A block takes eight neighbouring heads (or parts of fewer heads' tokens), a
// warp to each: with 8 KV heads a token's whole row is one run of memory.  One
// warp fetches by TMA, codes and pairs apart, five or six tiles of 32 tokens
// ahead; a block has the SM, so that a warp may keep 232 registers.
// Bound by how fast a warp's instructions follow one another: two warps a
// scheduler issue in 47% of the cycles, with the tensor cores 21% busy.  24
// requests of 32 heads (210 MB of codes and pairs) take 63 us, 3.4 TB/s; 100003
// tokens in groups of 32 channels (128 MB) 47 us.
#pragma once

#include "cg_attend.cuh"
#include "cg_quant.cuh"

namespace cg {

struct QuantArgs {
    uint32_t cols;       // code boxes of 128 bytes side by side in a tile
    uint32_t pw;         // bytes of a tile's pairs for one token
    uint32_t n_stages, stage, tile, ptile;  // tiles in flight; bytes of a stage, of a tile's codes of K, of its pairs of K
    float scale2;        // |scale| * log2 e, not 0
};

// Three warpgroups: two compute, one warp of the third fetches.  The launch gives 168 registers a thread, of which the
// third keeps 40 and the others take 232: 2 x 232 + 40 = 3 x 168.
constexpr uint32_t kQuantWarps = 8, kQuantThreads = 384, kQuantLens = 1024;
// Tokens that a warp takes at a time: 16 where a head's row has 128 bytes, else 32.
__host__ __device__ constexpr uint32_t quant_tok(uint32_t bits, uint32_t d) { return bits * d == 1024 ? 16 : 32; }
// Shared memory besides the stages: barriers, misc, lengths, and room to align.
constexpr uint32_t kQuantMaxStages = 8;
constexpr uint32_t kQuantMisc = 2 * kQuantMaxStages * 8, kQuantLensAt = kQuantMisc + 128;
constexpr uint32_t kQuantExtra = kQuantLensAt + kQuantLens * 4 + 1024;

// kN: column tiles of eight query rows.
#define CG_QUANT_ROWS(name)                                                                                             \
    cudaError_t name(uint32_t group, uint32_t n, const CUtensorMap &codes, const CUtensorMap &pairs, Args &a, const QuantArgs &q, \
                     int sms, cudaStream_t s)
CG_QUANT_ROWS(launch_quant_rows_4_64_f);
CG_QUANT_ROWS(launch_quant_rows_4_128_f);
CG_QUANT_ROWS(launch_quant_rows_8_64_f);
CG_QUANT_ROWS(launch_quant_rows_8_128_f);
CG_QUANT_ROWS(launch_quant_rows_4_64_b);
CG_QUANT_ROWS(launch_quant_rows_4_128_b);
CG_QUANT_ROWS(launch_quant_rows_8_64_b);
CG_QUANT_ROWS(launch_quant_rows_8_128_b);

#ifdef CG_QUANT_BITS
namespace {

__device__ __forceinline__ uint32_t pi(uint32_t x) { return x ^ ((x & 1u) << 2); }

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The i-th operand word of a word of codes: codes i and i + 4 of eight, or i and i + 2 of four.
template <uint32_t kBits> __device__ __forceinline__ uint32_t take(uint32_t w, uint32_t i) {
    if constexpr (kBits == 4) return ((i & 2u) ? w >> 8 : w) & ((i & 1u) ? 0x00F000F0u : 0x000F000Fu);
    return (i ? w >> 8 : w) & 0x00FF00FFu;
}

// kN words from shared memory at an address that is a multiple of their size (at most 16 bytes).
template <uint32_t kN> __device__ __forceinline__ void load_words(uint32_t (&w)[kN], uint32_t at) {
    if constexpr (kN == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
    if constexpr (kN == 2) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    if constexpr (kN == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
}
__device__ __forceinline__ uint32_t load_half(uint32_t at) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at));
    return x;
}

// Numbers of a pair, of type T.
template <class T> __device__ __forceinline__ float scale_of(uint32_t w) {
    if constexpr (__is_same(T, __half)) return __half2float(__ushort_as_half((uint16_t)w));
    return __uint_as_float(w << 16);
}
template <class T> __device__ __forceinline__ float low_of(uint32_t w) {
    if constexpr (__is_same(T, __half)) return __half2float(__ushort_as_half((uint16_t)(w >> 16)));
    return __uint_as_float(w & 0xFFFF0000u);
}
template <class T> __device__ __forceinline__ bool odd_pair(uint32_t w) {
    constexpr uint32_t kX = Half<T>::kExponent;
    return (w & kX) == kX || (w >> 16 & kX) == kX;
}
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b, float m, float n) {
    asm("{\n\t.reg .b64 s, t, v;\n\tmov.b64 s, {%2, %3};\n\tmov.b64 t, {%4, %5};\n\t"
        "mul.rn.f32x2 v, s, t;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "=f"(x), "=f"(y)
        : "f"(a), "f"(b), "f"(m), "f"(n));
}
// (x, y) += (a m, b n)
__device__ __forceinline__ void vfma2(float &x, float &y, float a, float b, float m, float n) {
    asm("{\n\t.reg .b64 s, t, u, v;\n\tmov.b64 s, {%2, %3};\n\tmov.b64 t, {%4, %5};\n\tmov.b64 u, {%0, %1};\n\t"
        "fma.rn.f32x2 v, s, t, u;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b), "f"(m), "f"(n));
}
// The power of two 2^e, e within -120 .. 120.
__device__ __forceinline__ float power2(int e) { return __uint_as_float((uint32_t)(127 + max(-120, min(120, e))) << 23); }
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 255u) - 127; }

template <class T, uint32_t kBits, uint32_t D, uint32_t G, uint32_t kN>
__global__ void __launch_bounds__(kQuantThreads, 1)
    k_quant_rows(const __grid_constant__ CUtensorMap codes, const __grid_constant__ CUtensorMap pairs, const Args a,
                 const QuantArgs qa) {
    constexpr uint32_t kTok = quant_tok(kBits, D), NG = D / G;
    constexpr uint32_t kHead = D * kBits / 8;              // bytes of a head's codes of a token
    constexpr uint32_t kGroup = G * kBits / 8;             // of a group's
    constexpr uint32_t kQuarter = kGroup / 4, kEighth = kGroup / 8;
    constexpr uint32_t kKWords = kQuarter / 4;             // words of a lane's quarter of a group
    constexpr bool kHalf = __is_same(T, __half);
    constexpr float kMiddle = kBits == 4 ? 8.f : 128.f;
    // What the sums of q are multiplied by: at most 128 2^15 2^-8 lies within fp16; bf16 ones are at once in the units of the
    // codes' part, so that a low value of 2^127 does not take the product past fp32.
    constexpr float kSumUnit = kHalf ? 0x1p-8f : 0x1p-24f;
    // Octaves that a weight may rise above the maximum that the sums go by.  Times low values they have to stay within fp32:
    // fp16's are below 2^16, bf16's may have any size.
    constexpr float kClimb = kHalf ? 60.f : 16.f;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (s_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm = s_addr(smem);
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    uint8_t *after = smem + qa.n_stages * qa.stage;
    const uint32_t full = s_addr(after), empty = full + 8 * kQuantMaxStages;
    if (tid == 0) {
        for (uint32_t k = 0; k < qa.n_stages; k++) {
            bar_init(full + 8 * k, 1);
            bar_init(empty + 8 * k, kQuantWarps);
        }
        fence_bar_init();
    }
    Walk w = take_share<kQuantThreads, true>(a, reinterpret_cast<uint64_t *>(after + kQuantMisc),
                                       reinterpret_cast<uint32_t *>(after + kQuantLensAt), kQuantLens);

    const uint32_t tt = 1u << a.tlog;  // tokens of a tile
    Piece p;
    uint32_t st = 0, phase = 0;        // stage of the next tile, and the parity of its barriers
    auto step = [&]() {
        if (++st == qa.n_stages) {
            st = 0;
            phase ^= 1u;
        }
    };
    if (warp >= kQuantWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp > kQuantWarps) return;
        // boxes of up to 2^rlog tokens of one block, K and V: `cols` of codes, one of pairs
        const uint32_t rlog = min(a.bshift, a.tlog), slog = a.tlog - rlog, subs = 1u << slog;
        const uint32_t boxes = 2u * subs * (qa.cols + 1);
        const uint32_t off = lane < subs ? lane << rlog : 0u;
        bool ok = true;
        uint32_t it = 0;
        while (ok && next_piece<true>(a, w, p)) {
            const bool shared = p.r == a.R;
            const uint32_t slot = shared ? a.shared_slot : a.slots ? a.slots[p.r] : p.r;
            const uint32_t *row = a.tables + (uint64_t)slot * a.n_blocks;
            const int x = (int)(p.group * a.nh * (kHead / 2)), xp = (int)((p.group * a.nh * NG * 2) & ~7u);
            uint32_t pos = (shared ? 0u : a.P) + (p.tile0 << a.tlog) + off;
            // the block of this lane's run; one past the sequence lies outside the maps and reads zeros
            uint32_t next = lane < subs && pos < p.len ? row[pos >> a.bshift] : a.n_pool;
            for (uint32_t k = 0; k < p.n; k++, it++, pos += tt) {
                uint32_t id = next;
                next = lane < subs && pos + tt < p.len && k + 1 < p.n ? row[(pos + tt) >> a.bshift] : a.n_pool;
                if (it >= qa.n_stages) ok = bar_wait(empty + 8 * st, phase ^ 1u);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                if (lane == 0) bar_expect(full + 8 * st, 2 * (qa.tile + qa.ptile));
                if (id > a.n_pool || (id == a.n_pool && lane < subs && pos < p.len)) {
                    id = a.n_pool;
                    flag(a.status, CG_ERR_RANGE);
                }
                __syncwarp();
                const uint32_t in = pos & ((1u << a.bshift) - 1u), base = sm + st * qa.stage;
                for (uint32_t b0 = 0; b0 < boxes; b0 += 32) {
                    const uint32_t b = b0 + lane, sub = b & (subs - 1u), kv = (b >> slog) & 1u, col = b >> (slog + 1);
                    const uint32_t bid = __shfl_sync(kFull, id, sub), bin = __shfl_sync(kFull, in, sub);
                    if (b >= boxes) continue;
                    if (col < qa.cols)
                        tma_box(base + kv * qa.tile + ((col << a.tlog) + (sub << rlog)) * 128, &codes, x + (int)col * 64, (int)bin,
                                (int)bid, (int)kv, full + 8 * st);
                    else
                        tma_box(base + 2 * qa.tile + kv * qa.ptile + (sub << rlog) * qa.pw, &pairs, xp, (int)bin, (int)bid,
                                (int)kv, full + 8 * st);
                }
                step();
            }
        }
        if (!ok) {  // wait for the copies in flight before leaving
            const uint32_t n = min(it, qa.n_stages);
            for (uint32_t k = 0; k < n; k++) {
                if (st == 0) {
                    st = qa.n_stages;
                    phase ^= 1u;
                }
                st--;
                bar_wait(full + 8 * st, phase);
            }
            if (lane == 0) flag_why(a.status, CG_ERR_TIMEOUT, kWhyWait);
        }
        if (a.pairs) wait_for_previous();  // this kernel is complete only after k_shared, whose pieces the joins read
        return;
    }

    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    let_next_start();
    const uint32_t c = lane & 3u, r = lane >> 2;
    const uint32_t hd = warp & (a.nh - 1u), part = warp >> a.hlog;  // head of the group, kTok tokens of the tile
    // This lane's places in a tile: rows pi(r) and on for K, tokens 2c, pi(2c + 1) and on for V; bits 4..6 of an
    // address are swizzled by its bits 7..9
    const uint32_t col = hd * kHead / 128, inner = hd * kHead % 128;
    const uint32_t tk = pi(r), t0 = 2 * c, t1 = pi(2 * c + 1);
    const uint32_t tile0 = sm + ((col << a.tlog) + part * kTok) * 128;
    // of the first group; the next group's address differs in bits 4..6 alone
    const uint32_t at_k = tile0 + tk * 128 + ((inner + c * kQuarter) ^ (tk << 4));
    const uint32_t at_v0 = tile0 + qa.tile + t0 * 128 + ((inner + r * kEighth) ^ (t0 << 4));
    const uint32_t at_v1 = tile0 + qa.tile + t1 * 128 + ((inner + r * kEighth) ^ (t1 << 4));
    // The queries of a piece, as they lie in memory, and how many of the item's tokens this lane's rows see.  They are
    // fetched before the results of the piece before it go out.
    uint4 raw[kN][D / 32];
    uint32_t sees[kN];
    auto fetch_queries = [&]() {
        const uint32_t head = p.group * a.nh + hd, own = p.r == a.R ? a.P : p.len - a.P;
#pragma unroll
        for (uint32_t n = 0; n < kN; n++) {
            const Row o = row_of(a, p, (p.range << a.rlog) + 8 * n + r, head < a.Hkv ? head : 0u);
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + o.r * a.qs[0] + o.i * a.qs[1] + o.h * a.qs[2]);
#pragma unroll
            for (uint32_t g = 0; g < NG; g++)
#pragma unroll
                for (uint32_t e = 0; e < G / 32; e++)
                    raw[n][g * (G / 32) + e] = o.valid ? src[g * (G / 8) + c * (G / 32) + e] : make_uint4(0, 0, 0, 0);
            sees[n] = own;
            if (p.r != a.R) {
                const uint32_t y = p.len + 1 + o.i;
                sees[n] = y > a.nq + a.P ? min(y - a.nq - a.P, own) : 0u;
            }
        }
    };
    bool ok = true, more = next_piece<true>(a, w, p);
    if (more) fetch_queries();
    while (more) {
        const bool shared = p.r == a.R, active = p.group * a.nh + hd < a.Hkv;
        const uint32_t own_tokens = shared ? a.P : p.len - a.P;
        const uint32_t pair0 = sm + 2 * qa.tile + ((p.group * a.nh * NG * 4) & 15u) + hd * NG * 4 + (part * kTok + tk) * qa.pw;
        uint32_t least = own_tokens;
        if (!shared) least = min(least, p.len + 1 > a.nq + a.P ? p.len + 1 - a.nq - a.P : 0u);
        // The queries, each scaled by a power of two so that its largest channel lies in [2^14, 2^15): bf16 ones then
        // become fp16, and parts 2^-25 of the largest and smaller lose bits.  qs: the sums of a query's channels over
        // lane c's group (c mod NG), in 16-bit parts with the pairs' type: 22 bits of fp16, 24 of bf16.
        constexpr uint32_t kSets = 4 / NG, kParts = kHalf ? 2 : 3, kLowMma = (kParts + 2 * kSets - 1) / (2 * kSets);
        uint32_t q[kN][D / 8], qs[kN][kLowMma][2], lim[kN][2];
        float fq[kN][2];
#pragma unroll
        for (uint32_t n = 0; n < kN; n++) {
            float x[D / 4], mx = 0.f;
#pragma unroll
            for (uint32_t e = 0; e < D / 32; e++) {
                const uint32_t v[4] = {raw[n][e].x, raw[n][e].y, raw[n][e].z, raw[n][e].w};
#pragma unroll
                for (uint32_t k = 0; k < 4; k++) {
                    const float2 y = Half<T>::unpack(v[k]);
                    x[8 * e + 2 * k] = y.x;
                    x[8 * e + 2 * k + 1] = y.y;
                    mx = fmaxf(mx, fmaxf(fabsf(y.x), fabsf(y.y)));
                }
            }
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            // (bf16's exponents go further than one factor: -113 .. 141)
            const int up = mx == 0.f || mx == INFINITY ? 0 : 14 - exponent(mx), up0 = kHalf ? up : up / 2;
            const float high = a.flip ? -power2(up0) : power2(up0);  // a negative scale turns q
#pragma unroll
            for (uint32_t e = 0; e < D / 4; e++) x[e] *= high;
            if constexpr (!kHalf) {
                const float rest = power2(up - up0);
#pragma unroll
                for (uint32_t e = 0; e < D / 4; e++) x[e] *= rest;
            }
            float sum = 0.f;
#pragma unroll
            for (uint32_t g = 0; g < NG; g++) {
                float y = 0.f;
#pragma unroll
                for (uint32_t e = 0; e < G / 4; e++) y += x[g * (G / 4) + e];
                y += __shfl_xor_sync(kFull, y, 1);
                y += __shfl_xor_sync(kFull, y, 2);
                if (g == (c & (NG - 1))) sum = y * kSumUnit;
            }
#pragma unroll
            for (uint32_t k = 0; k < kLowMma; k++) qs[n][k][0] = qs[n][k][1] = 0u;
#pragma unroll
            for (uint32_t k = 0; k < kParts; k++) {  // part k: set k mod kSets of operand word k / kSets
                const uint32_t y = Half<T>::pack(0.f, sum);
                if (c / NG == k % kSets) qs[n][k / kSets / 2][k / kSets % 2] = y;
                sum -= Half<T>::unpack(y).y;
            }
            constexpr uint32_t kPer = kBits == 4 ? 8 : 4;  // channels of a word
#pragma unroll
            for (uint32_t e = 0; e < D / 8; e++) {
                const uint32_t word = e / (kPer / 2), i = e % (kPer / 2), at = word * kPer + i;
                const float f = kBits == 4 && (i & 1u) ? 0.0625f : 1.f;
                q[n][e] = Half<__half>::pack(x[at] * f, x[at + kPer / 2] * f);
            }
            // what this lane's columns need, from the lanes that have the row
            // (neither 0 nor infinite: masked scores are -inf, and a score may be 0)
            const int down = 24 - up, down0 = down / 2;
            const float f = fminf(fmaxf(qa.scale2 * power2(down0) * power2(down - down0), 0x1p-149f), 0x1p127f);
#pragma unroll
            for (uint32_t j = 0; j < 2; j++) {
                const uint32_t from = (2 * c + j) * 4;
                fq[n][j] = __shfl_sync(kFull, f, from);
                lim[n][j] = __shfl_sync(kFull, sees[n], from);
            }
        }

        // Running maximum m and sum l of the weights, their products with the low values, and the power of two F that a
        // group's weights times scales are multiplied by before they become operands.
        // Codes are taken about their middle: the operands' rounding then meets half the codes' size, and the middle's part
        // is a product of its own (mid), taken away again at the end.  With two column tiles, whose registers spill, this is
        // done for fp16 and up to two groups a head: 40 rows of eight heads, groups of 64, are off by 2.5e-4 instead of 4.0e-4
        // (the output's own rounding: 2.1e-4), and with groups of 128 over 4000 tokens take 76 to 82 us instead of 75.  With
        // four groups it would be 136 instead of 103 us; bf16's output rounding, 1.7e-3, hides it (53 instead of 50 us).
        constexpr bool kMid = kN == 1 || (__is_same(T, __half) && NG <= 2);
        float o[kN][D / 16][4], m[kN][2], l[kN][2][2], lows[kN][NG][2][2], F[kN][NG][2][2], mid[kN][NG][4], most[NG];
#pragma unroll
        for (uint32_t g = 0; g < NG; g++) most[g] = 1.f;  // the larger F of the columns
#pragma unroll
        for (uint32_t n = 0; n < kN; n++) {
#pragma unroll
            for (uint32_t d = 0; d < D / 16; d++)
#pragma unroll
                for (uint32_t k = 0; k < 4; k++) o[n][d][k] = 0.f;
#pragma unroll
            for (uint32_t j = 0; j < 2; j++) {
                m[n][j] = -INFINITY;
                l[n][j][0] = l[n][j][1] = 0.f;
#pragma unroll
                for (uint32_t g = 0; g < NG; g++) {
                    lows[n][g][j][0] = lows[n][g][j][1] = 0.f;
                    F[n][g][j][0] = F[n][g][j][1] = 1.f;
                    mid[n][g][j] = mid[n][g][2 + j] = 0.f;
                }
            }
        }

        for (uint32_t k = 0; k < p.n; k++) {
            if (ok) ok = bar_wait(full + 8 * st, phase);
            if (!__all_sync(kFull, ok)) {
                ok = false;
                continue;
            }
            const uint32_t tok = ((p.tile0 + k) << a.tlog) + kTok * part;  // this warp's first token of the item
            const uint32_t base = st * qa.stage;
            // 16 tokens at a time; not unrolled: the loop's body alone fills the instruction cache
#pragma unroll 1
            for (uint32_t t = 0; active && t < kTok && tok + t < own_tokens; t += 16) {
                const uint32_t kp = base + pair0 + t * qa.pw, vp = kp + qa.ptile;
                const uint32_t kc = base + at_k + t * 128, vc0 = base + at_v0 + t * 128, vc1 = base + at_v1 + t * 128;
                const bool hidden = tok + t + 16 > least;  // some rows do not see some of the tokens, or there are none
                float s[kN][4], x[kN][2][2];  // scores; weights by column and row
                {
                    uint32_t pw[2][NG];
#pragma unroll
                    for (uint32_t h = 0; h < 2; h++) load_words<NG>(pw[h], kp + 8 * h * qa.pw);
                    // low values: words (scale, low) times (0, part of the sum of q)
                    uint32_t lo[2];
#pragma unroll
                    for (uint32_t h = 0; h < 2; h++) {
                        uint32_t y[1] = {pw[h][0]};
                        if constexpr (NG > 1) load_words<1>(y, kp + 8 * h * qa.pw + 4 * (c & (NG - 1)));
                        lo[h] = y[0];
                    }
                    const uint32_t lw[4] = {lo[0] & 0xFFFF0000u, lo[1] & 0xFFFF0000u, lo[0] & 0xFFFF0000u, lo[1] & 0xFFFF0000u};
#pragma unroll
                    for (uint32_t n = 0; n < kN; n++) {
                        Half<T>::mma0(s[n], lw, qs[n][0][0], qs[n][0][1]);
#pragma unroll
                        for (uint32_t e = 1; e < kLowMma; e++) Half<T>::mma(s[n], lw, qs[n][e][0], qs[n][e][1]);
                        if constexpr (kHalf)  // to the units of the codes' part
#pragma unroll
                            for (uint32_t e = 0; e < 4; e++) s[n][e] *= 0x1p-24f / kSumUnit;
                    }
                    constexpr uint32_t kChains = G >= 64 ? 2 : 1;  // sums of a group side by side
#pragma unroll
                    for (uint32_t g = 0; g < NG; g++) {
                        uint32_t wk[2][kKWords];
#pragma unroll
                        for (uint32_t h = 0; h < 2; h++) {
                            const uint32_t row = (kc ^ (g * kGroup)) + 8 * 128 * h;
                            if constexpr (kKWords == 8) {
                                uint32_t y[4], z[4];
                                load_words<4>(y, row);
                                load_words<4>(z, row ^ 16);
#pragma unroll
                                for (uint32_t e = 0; e < 4; e++) wk[h][e] = y[e], wk[h][4 + e] = z[e];
                            } else {
                                load_words<kKWords>(wk[h], row);
                            }
                        }
                        float acc[kN][kChains][4];
#pragma unroll
                        for (uint32_t e = 0; e < G / 16; e++) {
                            const uint32_t word = kBits == 4 ? e / 2 : e, i = kBits == 4 ? 2 * (e & 1u) : 0u;
                            const uint32_t x[4] = {take<kBits>(wk[0][word], i), take<kBits>(wk[1][word], i),
                                                   take<kBits>(wk[0][word], i + 1), take<kBits>(wk[1][word], i + 1)};
#pragma unroll
                            for (uint32_t n = 0; n < kN; n++) {
                                const uint32_t q0 = q[n][g * (G / 8) + 2 * e], q1 = q[n][g * (G / 8) + 2 * e + 1];
                                if (e < kChains) Half<__half>::mma0(acc[n][e % kChains], x, q0, q1);
                                else Half<__half>::mma(acc[n][e % kChains], x, q0, q1);
                            }
                        }
                        const float sc[2] = {scale_of<T>(pw[0][g]), scale_of<T>(pw[1][g])};
#pragma unroll
                        for (uint32_t n = 0; n < kN; n++)
#pragma unroll
                            for (uint32_t e = 0; e < 4; e++) {
                                const float y = kChains == 2 ? acc[n][0][e] + acc[n][kChains - 1][e] : acc[n][0][e];
                                s[n][e] = fmaf(y, sc[e >> 1], s[n][e]);
                            }
                    }
                }
                uint32_t pv[2][NG];  // the pairs of V
#pragma unroll
                for (uint32_t h = 0; h < 2; h++) load_words<NG>(pv[h], vp + 8 * h * qa.pw);
                if (hidden) {
#pragma unroll
                    for (uint32_t n = 0; n < kN; n++)
#pragma unroll
                        for (uint32_t e = 0; e < 4; e++)
                            if (tok + t + 4 * (e & 2u) + tk >= lim[n][e & 1u]) s[n][e] = -INFINITY;
#pragma unroll
                    for (uint32_t h = 0; h < 2; h++)
                        if (tok + t + 8 * h + tk >= own_tokens)  // a token of nobody's: its pairs hold anything
#pragma unroll
                            for (uint32_t g = 0; g < NG; g++) pv[h][g] = 0;
                }
                // Weights are 2^{s fq - m}.  m and F stay while no operand can exceed 2^15, by a lane's largest weight, scale
                // and F, and no weight 2^kClimb (V may be zero, its scales too).  Otherwise m becomes the maximum of a column that
                // did exceed it and F such that its largest operand lies in [2^4, 2^5), and O is scaled along: eleven octaves
                // go by before the next time.
                float widest = 0.f, x_most = -INFINITY;
#pragma unroll
                for (uint32_t g = 0; g < NG; g++) widest = fmaxf(widest, scale_of<T>(__vmaxu2(pv[0][g], pv[1][g])) * most[g]);
#pragma unroll
                for (uint32_t n = 0; n < kN; n++)
#pragma unroll
                    for (uint32_t j = 0; j < 2; j++) x_most = fmaxf(x_most, fmaf(fmaxf(s[n][j], s[n][2 + j]), fq[n][j], -m[n][j]));
                if (__builtin_expect(__any_sync(kFull, !(ex2(x_most) * widest <= 32768.f) || x_most > kClimb), 0)) {
#pragma unroll
                    for (uint32_t g = 0; g < NG; g++) most[g] = 0.f;
#pragma unroll
                    for (uint32_t n = 0; n < kN; n++)
#pragma unroll
                        for (uint32_t j = 0; j < 2; j++) {
                            const float y[2] = {s[n][j] * fq[n][j], s[n][2 + j] * fq[n][j]};
                            float mx = fmaxf(y[0], y[1]);
#pragma unroll
                            for (uint32_t d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                            // weights and their like against the maximum that m may become, fc of what they were
                            const float top = fmaxf(m[n][j], mx), z = top == -INFINITY ? 0.f : top;
                            const float fc = m[n][j] == top ? 1.f : ex2(m[n][j] - top), wt[2] = {ex2(y[0] - z), ex2(y[1] - z)};
                            float v[NG];  // the largest weights times scales
                            bool move = m[n][j] == -INFINITY ? mx != -INFINITY : mx > m[n][j] + kClimb;
#pragma unroll
                            for (uint32_t g = 0; g < NG; g++) {
                                v[g] = 0.f;
#pragma unroll
                                for (uint32_t h = 0; h < 2; h++)
                                    if (wt[h] != 0.f) v[g] = fmaxf(v[g], wt[h] * scale_of<T>(pv[h][g]));
#pragma unroll
                                for (uint32_t d = 4; d < 32; d <<= 1) v[g] = fmaxf(v[g], __shfl_xor_sync(kFull, v[g], d));
                                move |= v[g] * F[n][g][j][0] > 32768.f * fc;
                            }
                            // (a column moves for its own sake only: no query's rounding depends on the others)
                            const float f = move ? fc : 1.f;
                            if (move) m[n][j] = top;
                            l[n][j][0] *= f;
                            l[n][j][1] *= f;
#pragma unroll
                            for (uint32_t g = 0; g < NG; g++) {
                                float *F_ = F[n][g][j];
                                const float old = f / F_[0], nf = move ? power2(4 - exponent(fmaxf(v[g], 32.f * old))) : F_[0];
                                const float by = old * nf;
                                F_[0] = F_[1] = nf;
                                most[g] = fmaxf(most[g], nf);
                                lows[n][g][j][0] *= f;
                                lows[n][g][j][1] *= f;
#pragma unroll
                                for (uint32_t d = 0; d < G / 16; d++) {
                                    o[n][g * (G / 16) + d][j] *= by;
                                    o[n][g * (G / 16) + d][2 + j] *= by;
                                }
                                if constexpr (kMid) mid[n][g][j] *= by;
                            }
                        }
                }
#pragma unroll
                for (uint32_t n = 0; n < kN; n++)
#pragma unroll
                    for (uint32_t j = 0; j < 2; j++) {
                        const float z = m[n][j] == -INFINITY ? 0.f : m[n][j];
#pragma unroll
                        for (uint32_t h = 0; h < 2; h++) x[n][j][h] = ex2(fmaf(s[n][2 * h + j], fq[n][j], -z));
                        add2(l[n][j][0], l[n][j][1], x[n][j][0], x[n][j][1]);
                    }
                // A pair that is not finite must stay out of the rows that do not see its token, whose weight is 0: the rows
                // that do get it (infinite or NaN, as it is) here, and the products a zero.
                if (hidden)
#pragma unroll
                    for (uint32_t h = 0; h < 2; h++)
#pragma unroll
                        for (uint32_t g = 0; g < NG; g++)
                            if (odd_pair<T>(pv[h][g])) {
#pragma unroll
                                for (uint32_t n = 0; n < kN; n++)
#pragma unroll
                                    for (uint32_t j = 0; j < 2; j++)
                                        if (x[n][j][h] != 0.f) lows[n][g][j][h] += scale_of<T>(pv[h][g]) + low_of<T>(pv[h][g]);
                                pv[h][g] = 0;
                            }
                // O += operands times codes of V
#pragma unroll
                for (uint32_t g = 0; g < NG; g++) {
                    uint32_t b[kN][2];
                    const float sc[2] = {scale_of<T>(pv[0][g]), scale_of<T>(pv[1][g])};
                    float low[2] = {low_of<T>(pv[0][g]), low_of<T>(pv[1][g])};
                    if constexpr (kMid) {
                        low[0] = fmaf(sc[0], kMiddle, low[0]);
                        low[1] = fmaf(sc[1], kMiddle, low[1]);
                    }
#pragma unroll
                    for (uint32_t n = 0; n < kN; n++) {
                        float y[2][2];
#pragma unroll
                        for (uint32_t j = 0; j < 2; j++) {
                            // (in this order: a weight of 0 times a scale is not lost in an overflow)
                            mul2(y[j][0], y[j][1], x[n][j][0], x[n][j][1], sc[0], sc[1]);
                            mul2(y[j][0], y[j][1], y[j][0], y[j][1], F[n][g][j][0], F[n][g][j][1]);
                            vfma2(lows[n][g][j][0], lows[n][g][j][1], x[n][j][0], x[n][j][1], low[0], low[1]);
                        }
                        b[n][0] = transpose8(Half<__half>::pack(y[0][0], y[1][0]));
                        b[n][1] = transpose8(Half<__half>::pack(y[0][1], y[1][1]));
                        if constexpr (kMid) {
                            constexpr uint32_t k2 = (uint32_t)kMiddle * 0x10001u;
                            const uint32_t middles[4] = {k2, k2, k2, k2};
                            Half<__half>::mma(mid[n][g], middles, b[n][0], b[n][1]);
                        }
                    }
                    const uint32_t v0 = vc0 ^ (g * kGroup), v1 = vc1 ^ (g * kGroup), from[4] = {v0, v1, v0 + 8 * 128, v1 + 8 * 128};
                    constexpr uint32_t kWords = kEighth < 4 ? 1 : kEighth / 4;
                    uint32_t wv[4][kWords];
#pragma unroll
                    for (uint32_t e = 0; e < 4; e++) {
                        if constexpr (kEighth == 2) wv[e][0] = load_half(from[e]);
                        else load_words<kWords>(wv[e], from[e]);
                    }
                    // words of two tokens' codes side by side: channel by channel, operands along the tokens
                    constexpr uint32_t kHalves = kEighth < 4 ? 1 : 2 * kWords, kTiles = kBits == 4 ? 2 : 1;
#pragma unroll
                    for (uint32_t e = 0; e < kHalves; e++) {
                        const uint32_t sel = e & 1u ? 0x7632u : 0x5410u;
                        const uint32_t y0 = __byte_perm(wv[0][e / 2], wv[1][e / 2], sel), y1 = __byte_perm(wv[2][e / 2], wv[3][e / 2], sel);
#pragma unroll
                        for (uint32_t d = 0; d < kTiles; d++) {
                            const uint32_t v[4] = {take<kBits>(y0, 2 * d), take<kBits>(y0, 2 * d + 1), take<kBits>(y1, 2 * d),
                                                   take<kBits>(y1, 2 * d + 1)};
#pragma unroll
                            for (uint32_t n = 0; n < kN; n++)
                                Half<__half>::mma(o[n][g * (G / 16) + e * kTiles + d], v, b[n][0], b[n][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) bar_arrive(empty + 8 * st);
            step();
        }

        const Piece done = p;
        more = next_piece<true>(a, w, p);
        if (more) fetch_queries();
        if (active) {
            const bool answer = a.P == 0 && a.hlog == columns_log<true>() && done.n == done.of;  // the whole sequence
            const uint64_t slot = a.part0 + ((((uint64_t)blockIdx.x + done.item) << columns_log<true>()) + warp) * a.piece_rows;
            const uint32_t head = done.group * a.nh + hd, row0 = done.range << a.rlog;
#pragma unroll
            for (uint32_t n = 0; n < kN; n++)
#pragma unroll
                for (uint32_t j = 0; j < 2; j++) {
                    float sum = l[n][j][0] + l[n][j][1], low[NG];
#pragma unroll
                    for (uint32_t g = 0; g < NG; g++) low[g] = lows[n][g][j][0] + lows[n][g][j][1];
#pragma unroll
                    for (uint32_t d = 4; d < 32; d <<= 1) {
                        sum += __shfl_xor_sync(kFull, sum, d);
#pragma unroll
                        for (uint32_t g = 0; g < NG; g++) low[g] += __shfl_xor_sync(kFull, low[g], d);
                    }
                    const uint32_t x = 8 * n + 2 * c + j;
                    const Row row = row_of(a, done, row0 + x, head);
                    if (!row.valid) continue;
                    const float inv = !answer ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
                    float *part_o = a.part_o + (slot + x) * D;
                    uint16_t *dst = a.out + row.r * a.os[0] + row.i * a.os[1] + row.h * a.os[2];
                    constexpr uint32_t kPer = G / 8;  // channels of a group that this lane has
#pragma unroll
                    for (uint32_t g = 0; g < NG; g++) {
                        // (two factors: their product may lie past fp32 where V is large)
                        const float unit = 1.f / F[n][g][j][0], centre = kMid ? mid[n][g][j] : 0.f;
                        float y[kPer];
#pragma unroll
                        for (uint32_t d = 0; d < kPer / 2; d++) {
                            y[2 * d] = fmaf((o[n][g * (G / 16) + d][j] - centre) * 0x1p24f, unit, low[g]) * inv;
                            y[2 * d + 1] = fmaf((o[n][g * (G / 16) + d][2 + j] * (kBits == 4 ? 0.0625f : 1.f) - centre) * 0x1p24f, unit, low[g]) * inv;
                        }
                        const uint32_t ch = g * G + r * kPer;
                        if (answer) {
#pragma unroll
                            for (uint32_t d = 0; d < kPer; d += 4) {
                                *reinterpret_cast<uint2 *>(dst + ch + d) = make_uint2(Half<T>::pack(y[d], y[d + 1]), Half<T>::pack(y[d + 2], y[d + 3]));
                            }
                        } else {
#pragma unroll
                            for (uint32_t d = 0; d < kPer; d += 4)
                                *reinterpret_cast<float4 *>(part_o + ch + d) = make_float4(y[d], y[d + 1], y[d + 2], y[d + 3]);
                        }
                    }
                    if (r == 0) {
                        if (!answer) a.part_ml[slot + x] = make_float2(m[n][j], sum);
                        else if (a.lse)
                            a.lse[((uint64_t)row.r * a.nq + row.i) * (a.g * a.Hkv) + row.h] =
                                sum == 0.f ? -INFINITY : (m[n][j] + log2f(sum)) * 0.6931471805599453f;
                    }
                }
        }
    }
    if (!ok && lane == 0) flag_why(a.status, CG_ERR_TIMEOUT, kWhyWait);
}

template <class T, uint32_t kBits, uint32_t D, uint32_t G, uint32_t kN>
CG_QUANT_ROWS(launch_one) {
    const uint32_t bytes = q.n_stages * q.stage + kQuantExtra;
    const auto k = k_quant_rows<T, kBits, D, G, kN>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    a.n_cta = (uint32_t)sms < kMaxCtas ? sms : kMaxCtas;
    return launch_next(k, a.n_cta, kQuantThreads, bytes, s, a.pairs != 0, codes, pairs, a, q);
}
template <class T, uint32_t kBits, uint32_t D, uint32_t G>
CG_QUANT_ROWS(launch_group) {
    return n == 1 ? launch_one<T, kBits, D, G, 1>(group, n, codes, pairs, a, q, sms, s)
                  : launch_one<T, kBits, D, G, 2>(group, n, codes, pairs, a, q, sms, s);
}
template <class T, uint32_t kBits, uint32_t D>
CG_QUANT_ROWS(launch_rows) {
    if constexpr (D == 128)
        if (group == 128) return launch_group<T, kBits, D, 128>(group, n, codes, pairs, a, q, sms, s);
    return group == 64 ? launch_group<T, kBits, D, 64>(group, n, codes, pairs, a, q, sms, s)
                       : launch_group<T, kBits, D, 32>(group, n, codes, pairs, a, q, sms, s);
}

}  // namespace
#endif

}  // namespace cg
