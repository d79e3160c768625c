// kv4.cuh -- a paged KV cache held in 4 bits, and decode attention over it.
//
// Format.  A group is 32 consecutive elements of one head vector.  Its scale s is max|x| / 7
// rounded (to nearest, ties to even) to an unsigned 8-bit float with 5 exponent bits (bias 15)
// and 3 mantissa bits, at most 7680: the byte shifted left by 7 is the same number in fp16.  An
// element is c = clamp(rne(x / s), -7, 7), stored as c + 8 in 4 bits; a group that holds a NaN or an
// infinity gets the scale 0xFF (a NaN).  s * c has 7 significant bits at most, so bf16 and fp16
// hold it exactly, and the rounding to 4 bits (half a step, s / 2) is the only one.
//
// A record of 2176 bytes holds 16 consecutive rows of one KV head, K and V, so one bulk copy
// brings all that attention needs of them; the cache is uint8 [num_pages, Hkv, page_size / 16, 2176].
// Inside a record the codes lie in the order in which the lanes of a warp (g = lane / 4,
// t = lane % 4) feed them to mma.m16n8k16, so that every lane reads 16 consecutive bytes:
//   0    K codes   row r, chunk t (16 bytes at 64 r + 16 t): word w holds elements 16 s + 4 t + i, s = 2w, 2w + 1,
//                  at bit 16 (i % 2) + 4 (2 (s % 2) + i / 2)
//   1024 V codes   row r, piece g (8 bytes at 512 (r / 8) + 64 g + 16 (r % 8 / 2) + 8 (r % 2)): elements 16 g + k
//                  at bit 4 k
//   2048 K scales  [row][group]
//   2112 V scales  [group][row]
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "decode.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace gqa {

constexpr int kRec = 2176;         // bytes of a record
constexpr int kRecRows = 16;       // rows of a record
constexpr int kRecV = 1024;        // V codes
constexpr int kRecKs = 2048;       // K scales
constexpr int kRecVs = 2112;       // V scales

// A kernel launched with programmatic stream serialization may start before the one ahead of it in its stream
// has ended: wait for that one (and the visibility of its writes), and let the next one start likewise.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void mbar_inval(uint32_t bar) {
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A paged 4-bit cache: row r of sequence b is row r % 16 of record
// (table[b * max_pages + r / page_size] * Hkv + head) * (page_size / 16) + r % page_size / 16.
struct Kv4Cache {
    uint8_t *recs;
    const int32_t *table;
    int num_pages, page_size, max_pages, Hkv;
};

// Page that holds row r of sequence b, or -1 where the table names none.
__device__ __forceinline__ int kv4_page(const Kv4Cache &c, int b, long long row) {
    if (row < 0 || row >= static_cast<long long>(c.max_pages) * c.page_size) return -1;   // the product is below 2^31
    const int id = c.table[static_cast<size_t>(b) * c.max_pages + static_cast<int>(row) / c.page_size];
    return id >= 0 && id < c.num_pages ? id : -1;
}

__device__ __forceinline__ uint8_t *kv4_record(const Kv4Cache &c, int page, int head, int row_in_page) {
    const size_t i = (static_cast<size_t>(page) * c.Hkv + head) * (c.page_size / kRecRows) + row_in_page / kRecRows;
    return c.recs + i * kRec;
}

// ------------------------------------------------------------------ quantiser
// Scale byte of a group whose largest magnitude has the fp32 bit pattern amax (a bf16 number).
__device__ __forceinline__ uint32_t kv4_scale_byte(uint32_t amax) {
    const float a = __uint_as_float(amax);
    constexpr float kSeventh = 1.0f / 7.0f;
    float y = a * kSeventh;                           // a / 7, rounded as a division: a value halfway between two
    y = fmaf(fmaf(-7.0f, y, a), kSeventh, y);         // scales has few bits and comes out exactly
    // times 2^-112 the scale's exponent is the fp32 number's, subnormal ones included, and the byte its upper bits
    uint32_t u = __float_as_uint(y * 1.925929944387236e-34f);
    u = (u + 0x7ffffu + ((u >> 20) & 1u)) >> 20;
    return amax >= 0x7f800000u ? 0xffu : min(u, 223u);
}

__device__ __forceinline__ float kv4_scale(uint32_t byte) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// 1 / s as a sum of two floats: x * hi + x * lo, rounded once, is x / s rounded, so that a quotient
// halfway between two codes is met exactly.  0 for s = 0 and for a NaN.
__device__ __forceinline__ float2 kv4_inverse(float s) {
    float2 v = make_float2(0.f, 0.f);
    if (s > 0.f) {
        v.x = __fdiv_rn(1.0f, s);
        v.y = __fmaf_rn(-s, v.x, 1.0f) * v.x;
    }
    return v;
}

// |x / s| stays below 7.5 wherever the scale was rounded to 4 bits, up by 1/16 at most; it may not for smaller or
// larger groups.
__device__ __forceinline__ bool kv4_clamps(uint32_t byte) { return byte < 8u || byte >= 223u; }

// Codes of two elements as the bits of 2^23 * 1.5 + 8 + c: the sum rounds to a whole number, ties to even.
constexpr float kCodeMagic = 12582920.0f;
constexpr uint32_t kCodeMagicBits = 0x4b400000u;   // of 2^23 * 1.5
template <bool CLAMP>
__device__ __forceinline__ uint2 kv4_code2(uint32_t bf16x2, float2 inv) {
    const float2 x = make_float2(bf16lo(bf16x2), bf16hi(bf16x2));
    float2 r = __ffma2_rn(x, make_float2(inv.x, inv.x), __fmul2_rn(x, make_float2(inv.y, inv.y)));
    if constexpr (CLAMP) {
        r.x = fminf(fmaxf(r.x, -7.0f), 7.0f);
        r.y = fminf(fmaxf(r.y, -7.0f), 7.0f);
    }
    r = __fadd2_rn(r, make_float2(kCodeMagic, kCodeMagic));
    return make_uint2(__float_as_uint(r.x), __float_as_uint(r.y));
}
// c + 8 of one element.
__device__ __forceinline__ uint32_t kv4_code(float x, float2 inv) {
    const float r = fminf(fmaxf(__fmaf_rn(x, inv.x, x * inv.y), -7.0f), 7.0f);
    return __float_as_uint(r + kCodeMagic) & 15u;
}

// ------------------------------------------------------------------ bf16 rows <-> records
struct Kv4RowsParams {
    uint16_t *k, *v;          // bf16 [N, Hkv, D], rows k_stride / v_stride elements apart
    long long k_stride, v_stride;
    const int64_t *cu;        // [B + 1]
    const int32_t *prefix;    // [B]
    Kv4Cache cache;
    unsigned *err;
    long long N;
    unsigned units;
    unsigned parts;           // of a unit, `heads` heads each (the last may have fewer)
    int heads, B;
};

// The units of sequence b (16-row records of its rows prefix .. prefix + len - 1) are numbered from
// here on: at most len / 16 + 2 of them, so that no prefix sum over the sequences is needed.
__device__ __forceinline__ long long kv4_first_unit(const int64_t *cu, int b) { return cu[b] / kRecRows + 2ll * b; }

// The sequence that unit `unit` belongs to: the last one whose first unit is not behind it.  32 lanes look at
// a time.
__device__ __forceinline__ int kv4_sequence_of(const int64_t *cu, int B, long long unit, int lane) {
    int lo = 0, n = B;   // among lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32, b = lo + lane * step;
        const bool at = lane * step < n && (lane == 0 || kv4_first_unit(cu, b) <= unit);
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, at));
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Rows of K and V between bf16 and records: a warp takes a unit for some heads, eight rows of a head at a time.  Bound by
// memory: 512 B of bf16 and 136 B of record per row and head; every load and store of whole records is coalesced, and
// the loads of eight rows are issued together.  The unit's place is found once for its heads (four dependent
// loads); packed arithmetic and a table of the 256 inverse scales keep the quantiser below the memory's time.  68K tokens of
// 8 heads in and out: 137 us, 4.6 TB/s.
template <bool WRITE>
__global__ void __launch_bounds__(256, WRITE ? 4 : 5) kv4_rows_kernel(const __grid_constant__ Kv4RowsParams p) {
    __shared__ float2 s_inv[256];
    grid_dependency_wait();
    grid_dependents_launch();
    if constexpr (WRITE) {
        s_inv[threadIdx.x] = kv4_inverse(kv4_scale(threadIdx.x));
        __syncthreads();
    }
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    auto bounds_ok = [&](int b) {
        return p.cu[b] >= 0 && p.cu[b + 1] >= p.cu[b] && p.cu[b + 1] <= p.N && p.prefix[b] >= 0;
    };
    const unsigned w = blockIdx.x * 8 + (threadIdx.x >> 5);
    for (long long b = w * 32ll + lane; b < p.B; b += gridDim.x * 256ll)
        if (!bounds_ok(static_cast<int>(b))) atomicOr(p.err, kErrInput);
    const unsigned unit = w / p.parts;
    if (unit >= p.units) return;
    const int head0 = w % p.parts * p.heads, head1 = min(p.cache.Hkv, head0 + p.heads);
    const int b = kv4_sequence_of(p.cu, p.B, unit, lane);
    if (!bounds_ok(b) || unit < kv4_first_unit(p.cu, b)) return;
    const long long tok0 = p.cu[b], tok1 = p.cu[b + 1], r0 = p.prefix[b], r1 = r0 + (tok1 - tok0);   // rows r0 .. r1 - 1
    const long long base = (r0 / kRecRows + (unit - kv4_first_unit(p.cu, b))) * kRecRows;
    if (tok1 == tok0 || base >= r1) return;
    const int page = kv4_page(p.cache, b, base);
    if (page < 0) {
        if (head0 == 0 && lane == 0) atomicOr(p.err, kErrInput);
        if (WRITE) return;
    }
    const int rip = static_cast<int>(base % p.cache.page_size);
    const long long tok_of_row0 = tok0 - r0 + base;   // packed token of the record's row 0
    const int from = static_cast<int>(max(0ll, r0 - base)), till = static_cast<int>(min(16ll, r1 - base));
#pragma unroll 1
    for (int i = 2 * head0; i < 2 * head1; ++i) {
        const int head = i >> 1, hb = i & 1;   // rows 8 hb .. + 7
        uint8_t *rec = page < 0 ? nullptr : kv4_record(p.cache, page, head, rip);
        auto has = [&](int r) { return r >= from && r < till; };
        // K: lane (g, t) holds elements 16 s + 4 t .. + 3 of row 8 hb + g; V: elements 16 g .. + 15 of rows 8 hb + 2 t, + 1
        const int rk = 8 * hb + g, rv = 8 * hb + 2 * t;
        uint16_t *krow = p.k + (tok_of_row0 + rk) * p.k_stride + head * kHeadDim + 4 * t;
        uint16_t *vrow = p.v + (tok_of_row0 + rv) * p.v_stride + head * kHeadDim + 16 * g;
        if constexpr (WRITE) {
            uint2 x[8];
            uint4 y[2][2];
#pragma unroll
            for (int s = 0; s < 8; ++s) x[s] = has(rk) ? __ldg(reinterpret_cast<const uint2 *>(krow + 16 * s)) : make_uint2(0u, 0u);
#pragma unroll
            for (int par = 0; par < 2; ++par)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    y[par][e] = has(rv + par) ? __ldg(reinterpret_cast<const uint4 *>(vrow + par * p.v_stride) + e) : make_uint4(0u, 0u, 0u, 0u);
            uint32_t m[4];
#pragma unroll
            for (int wd = 0; wd < 4; ++wd) {
                m[wd] = __vmaxu2(__vmaxu2(x[2 * wd].x & 0x7fff7fffu, x[2 * wd].y & 0x7fff7fffu),
                                 __vmaxu2(x[2 * wd + 1].x & 0x7fff7fffu, x[2 * wd + 1].y & 0x7fff7fffu));
                m[wd] = __vmaxu2(m[wd], __shfl_xor_sync(0xffffffffu, m[wd], 1));
                m[wd] = __vmaxu2(m[wd], __shfl_xor_sync(0xffffffffu, m[wd], 2));
            }
            const uint32_t mine = t == 0 ? m[0] : t == 1 ? m[1] : t == 2 ? m[2] : m[3];   // lane t takes group t
            const uint32_t own = kv4_scale_byte(max(mine & 0xffffu, mine >> 16) << 16);
            uint32_t scales = own << (8 * t);
            scales |= __shfl_xor_sync(0xffffffffu, scales, 1);
            scales |= __shfl_xor_sync(0xffffffffu, scales, 2);
            uint32_t word[4];
            auto encode_k = [&](auto clamp) {
#pragma unroll
                for (int wd = 0; wd < 4; ++wd) {
                    const float2 inv = s_inv[(scales >> (8 * wd)) & 255u];
                    uint32_t u = 0u - kCodeMagicBits * 0x11111111u;
#pragma unroll
                    for (int o = 0; o < 2; ++o) {   // s = 2 wd + o
                        const uint2 a = kv4_code2<decltype(clamp)::value>(x[2 * wd + o].x, inv);
                        const uint2 c = kv4_code2<decltype(clamp)::value>(x[2 * wd + o].y, inv);
                        u += a.x * (1u << (8 * o)) + a.y * (1u << (8 * o + 16)) + c.x * (1u << (8 * o + 4)) + c.y * (1u << (8 * o + 20));
                    }
                    word[wd] = u;
                }
            };
            if (__any_sync(0xffffffffu, kv4_clamps(own)))
                encode_k(std::true_type{});
            else
                encode_k(std::false_type{});
            if (has(rk)) {
                *reinterpret_cast<uint4 *>(rec + 64 * rk + 16 * t) = make_uint4(word[0], word[1], word[2], word[3]);
                if (t == 0) *reinterpret_cast<uint32_t *>(rec + kRecKs + 4 * rk) = scales;
            }
            uint32_t byte[2], o[2][2];
#pragma unroll
            for (int par = 0; par < 2; ++par) {
                uint32_t mv = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    mv = __vmaxu2(mv, __vmaxu2(__vmaxu2(y[par][e].x & 0x7fff7fffu, y[par][e].y & 0x7fff7fffu),
                                               __vmaxu2(y[par][e].z & 0x7fff7fffu, y[par][e].w & 0x7fff7fffu)));
                mv = __vmaxu2(mv, __shfl_xor_sync(0xffffffffu, mv, 4));   // the group's other 16 elements
                byte[par] = kv4_scale_byte(max(mv & 0xffffu, mv >> 16) << 16);
            }
            auto encode_v = [&](auto clamp) {
#pragma unroll
                for (int par = 0; par < 2; ++par) {
                    const float2 inv = s_inv[byte[par]];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t z[4] = {y[par][h].x, y[par][h].y, y[par][h].z, y[par][h].w};
                        o[par][h] = 0u - kCodeMagicBits * 0x11111111u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint2 a = kv4_code2<decltype(clamp)::value>(z[e], inv);
                            o[par][h] += a.x * (1u << (8 * e)) + a.y * (1u << (8 * e + 4));
                        }
                    }
                }
            };
            if (__any_sync(0xffffffffu, kv4_clamps(byte[0]) || kv4_clamps(byte[1])))
                encode_v(std::true_type{});
            else
                encode_v(std::false_type{});
#pragma unroll
            for (int par = 0; par < 2; ++par)
                if (has(rv + par)) {
                    *reinterpret_cast<uint2 *>(rec + kRecV + 512 * hb + 16 * lane + 8 * par) = make_uint2(o[par][0], o[par][1]);
                    if ((g & 1) == 0) rec[kRecVs + 16 * (g >> 1) + rv + par] = static_cast<uint8_t>(byte[par]);
                }
        } else {
            // a code c' at bits 0..3 of 128.0 reads as 128 + c' in bf16: minus 136 it is c, times s the value, both exact
            uint4 kc = make_uint4(0u, 0u, 0u, 0u), vc = kc;
            uint32_t ks = 0, vs = 0;
            if (rec != nullptr) {
                kc = *reinterpret_cast<const uint4 *>(rec + 512 * hb + 16 * lane);
                vc = *reinterpret_cast<const uint4 *>(rec + kRecV + 512 * hb + 16 * lane);
                ks = *reinterpret_cast<const uint32_t *>(rec + kRecKs + 4 * rk);
                vs = *reinterpret_cast<const uint16_t *>(rec + kRecVs + 16 * (g >> 1) + rv);
            }
            auto bf16_scale = [](uint32_t byte) {   // in both halves
                return pack_bf16x2(kv4_scale(byte), kv4_scale(byte));
            };
            auto values = [](uint32_t codes, uint32_t scale) {   // codes at bits 0..3 of both halves
                const uint32_t c = (codes & 0x000f000fu) | 0x43004300u;
                uint32_t v;
                asm("{\n\t.reg .b32 d;\n\tadd.rn.bf16x2 d, %1, %2;\n\tmul.rn.bf16x2 %0, d, %3;\n\t}" : "=r"(v) : "r"(c), "r"(0xc308c308u), "r"(scale));
                return v;
            };
            const uint32_t word[4] = {kc.x, kc.y, kc.z, kc.w};
            if (has(rk))
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint32_t sc = bf16_scale((ks >> (8 * (s >> 1))) & 255u), u = word[s >> 1] >> (8 * (s & 1));
                    *reinterpret_cast<uint2 *>(krow + 16 * s) = make_uint2(values(u, sc), values(u >> 4, sc));
                }
#pragma unroll
            for (int par = 0; par < 2; ++par) {
                if (!has(rv + par)) continue;
                const uint32_t sc = bf16_scale((vs >> (8 * par)) & 255u);
                const uint32_t half[2] = {par ? vc.z : vc.x, par ? vc.w : vc.y};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t up = half[h] >> 4;
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = values(__byte_perm(half[h], up, 0x0400u + 0x0101u * e), sc);
                    reinterpret_cast<uint4 *>(vrow + par * p.v_stride)[h] = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ decode
struct Kv4DecodeParams {
    const uint16_t *q;        // bf16 [B, H, D]
    const uint16_t *k_new;    // bf16 [B, Hkv, D] (append)
    const uint16_t *v_new;
    Kv4Cache cache;
    const int32_t *seqlens;   // [B]
    const int32_t *qpos;      // [B] or nullptr (position = seqlens[b])
    const float *wq, *wk;     // [D]
    float *part_o;            // [slots, HG, D]
    float *part_ml;           // [slots, HG, 2]
    int2 *plan;               // [B * Hkv * passes]: first team of the pair, teams
    float *scores;            // [B * H, score_stride] base-2 logits, or nullptr
    long long score_stride;
    float *out;               // [B, H, D]
    unsigned *err;
    int B, H, hpg, passes, max_len;
    int len_add;              // 1 after an append
    int pairing;
    float eps;
    float scale_log2;
    uint32_t base0, base1;    // kCodeBase0, kCodeBase1 (see kv4_pick)
    RopeFreqs rf;
};

// len = seqlens[b] + len_add rows attended: 1 <= len <= max_len, within the table's pages.
__device__ __forceinline__ bool kv4_seq_ok(const Kv4DecodeParams &p, int b, int &len) {
    len = p.seqlens[b] + p.len_add;
    return len >= 1 && len <= p.max_len &&
           static_cast<long long>(len) <= static_cast<long long>(p.cache.max_pages) * p.cache.page_size;
}

// cos and sin in 64 bits (the appended key: see kv4_new_row).
__device__ __forceinline__ void kv4_rope4_f64(double (&a)[4], int pos, const RopeFreqs &rf, int pairing, int lane) {
    if (pairing == kPairAdjacent) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            double s, c;
            sincos(static_cast<double>(pos) * rf.inv_freq[2 * lane + k], &s, &c);
            const double x = a[2 * k], y = a[2 * k + 1];
            a[2 * k] = x * c - y * s;
            a[2 * k + 1] = x * s + y * c;
        }
    } else {
        const double sign = lane < 16 ? -1.0 : 1.0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const double o = __shfl_xor_sync(0xffffffffu, a[k], 16);
            double s, c;
            sincos(static_cast<double>(pos) * rf.inv_freq[4 * (lane & 15) + k], &s, &c);
            a[k] = a[k] * c + sign * o * s;
        }
    }
}

// Quantise and store one row of a record (in global and in shared memory), lane l holding elements 4 l .. 4 l + 3
// of K and V.
__device__ __forceinline__ void kv4_store_row(uint8_t *rec, int r, const float (&k)[4], const float (&v)[4], int lane) {
    const int s = lane >> 2, t = lane & 3;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float *x = which ? v : k;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t byte = kv4_scale_byte(m);
        const float2 inv = kv4_inverse(kv4_scale(byte));
        const uint32_t c0 = kv4_code(x[0], inv), c1 = kv4_code(x[1], inv), c2 = kv4_code(x[2], inv), c3 = kv4_code(x[3], inv);
        if (which == 0) {
            uint8_t *dst = rec + 64 * r + 16 * t + 4 * (s >> 1) + (s & 1);
            dst[0] = static_cast<uint8_t>(c0 | c2 << 4);
            dst[2] = static_cast<uint8_t>(c1 | c3 << 4);
            if ((lane & 7) == 0) rec[kRecKs + 4 * r + (lane >> 3)] = static_cast<uint8_t>(byte);
        } else {
            uint8_t *dst = rec + kRecV + 512 * (r >> 3) + 64 * s + 16 * ((r & 7) >> 1) + 8 * (r & 1) + 2 * t;
            *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(c0 | c1 << 4 | c2 << 8 | c3 << 12);
            if ((lane & 7) == 0) rec[kRecVs + 16 * (lane >> 3) + r] = static_cast<uint8_t>(byte);
        }
    }
}

// k-hat and v of the new token of (sequence b, KV head g), by one warp.  k-hat is evaluated in 64 bits and
// rounded to bf16 before the quantiser, so that the 4-bit row does not depend on the order of fp32 sums where a
// value lies next to a border between two codes.
__device__ __forceinline__ void kv4_new_row(const Kv4DecodeParams &p, int b, int g, float (&k)[4], float (&v)[4], int lane) {
    const size_t src = (static_cast<size_t>(b) * p.cache.Hkv + g) * kHeadDim + 4 * lane;
    const uint2 kr = *reinterpret_cast<const uint2 *>(p.k_new + src);
    const uint2 vr = *reinterpret_cast<const uint2 *>(p.v_new + src);
    const float x[4] = {bf16lo(kr.x), bf16hi(kr.x), bf16lo(kr.y), bf16hi(kr.y)};
    const float4 w4 = reinterpret_cast<const float4 *>(p.wk)[lane];
    const float w[4] = {w4.x, w4.y, w4.z, w4.w};
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) ss += static_cast<double>(x[i]) * x[i];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const double inv = 1.0 / sqrt(ss * (1.0 / kHeadDim) + static_cast<double>(p.eps));
    double y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = static_cast<double>(w[i]) * x[i] * inv;
    kv4_rope4_f64(y, p.qpos ? p.qpos[b] : p.seqlens[b], p.rf, p.pairing, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) k[i] = bf16lo(pack_bf16x2(static_cast<float>(y[i]), 0.f));
    v[0] = bf16lo(vr.x);
    v[1] = bf16hi(vr.x);
    v[2] = bf16lo(vr.y);
    v[3] = bf16hi(vr.y);
}

// D = A B + C, A 16 x 16 (fp16), B 16 x 8 (fp16), fp32 accumulation.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    mma16816(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}
// The 8 x 8 matrix of 16-bit elements whose row lane / 4 holds x in columns 2 (lane % 4) and + 1, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Two floats to fp16 (nearest even), `lo` in the low half, and what the rounding left over, rounded the same way:
// together 22 significant bits.
__device__ __forceinline__ void h2_split(float lo, float hi, uint32_t &h, uint32_t &rest) {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(hi - f.y), "f"(lo - f.x));
}

// Codes to fp16.  A code c' = c + 8 at bits 0..3 of 8.0 reads as 8 + c'/128, at bits 4..7 of 0.5 as 0.5 + c'/128.
// K: minus 8 + 8/128 or 0.5 + 8/128 that is c/128, and the group's scale multiplies its sum of products in fp32.
// V: its scales run along the summed rows, so they go into the elements: one fma with the scale and -(8 + 8/128) s or
// -(0.5 + 8/128) s gives s c / 128, without any rounding: 129 s and 9 s have at most 11 significant bits.
// The factor 1/128 keeps those products below fp16's largest number for every scale; it goes back into the logits' factor
// and the output.  (As subnormals, c' 2^-24 and c' 2^-20 by an AND alone, K's codes cost the products six bits: the
// matrix instruction aligns them as if they were normal.)
constexpr uint32_t kCodeMask0 = 0x000f000fu, kCodeMask1 = 0x00f000f0u;
constexpr uint32_t kCodeBase0 = 0x48004800u, kCodeBase1 = 0x38003800u;   // 8.0, 0.5
constexpr uint32_t kCodeOff0 = 0xc808c808u, kCodeOff1 = 0xb880b880u;     // -8.0625, -0.5625
constexpr float kCodeUnit = 128.0f;

// Softmax weights to fp16.  P = 2^(logit - m) with m moved up as soon as a logit exceeds it by more than kMaxAhead: P is at
// most 2^kMaxAhead, and 2^(15 - kMaxAhead) P at most 2^15.  As two fp16 numbers that product keeps 22 bits, or, where the
// second would be subnormal, all down to its step 2^-24: a weight is off by at most 2^-22 of itself or 2^-38 of the
// largest, whichever is more, so rows that weigh next to nothing still count by the thousand.  (Without the factor the step is
// 2^-24, and 8192 rows of 2^-25 beside one of 1 leave the output though l sums them.)  A smaller kMaxAhead would move m, and
// scale O, more often: normal logits of deviation 1 do so in 2 or 3 of a warp's 256 units at 2, in 17 at 0.  64 sequences
// of 1K to 32K rows take 230 us with the factor, 228 without.
constexpr float kMaxAhead = 2.0f;
constexpr float kWeightUnit = 8192.0f;   // 2^(15 - kMaxAhead)

struct Kv4Scale2 {
    uint32_t s, o0, o1;
};
// bytes: the scales of two rows in its two low bytes
__device__ __forceinline__ Kv4Scale2 kv4_scale2(uint32_t bytes) {
    Kv4Scale2 r;
    r.s = __byte_perm(bytes, 0u, 0x1404u) >> 1;   // each byte in the high byte of a half, then << 7 in place of << 8
    r.o0 = h2_mul(r.s, kCodeOff0);
    r.o1 = h2_mul(r.s, kCodeOff1);
    return r;
}
// (x & mask) | base in one instruction: that takes one immediate only, so base comes in a register (from the kernel's
// parameters; the compiler turns a constant into a second instruction for every operand).
template <uint32_t MASK>
__device__ __forceinline__ uint32_t kv4_pick(uint32_t x, uint32_t base) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(x), "n"(MASK), "r"(base));
    return d;
}
// The scales of groups 0, 2 and 1, 3 of a row as fp32.
__device__ __forceinline__ void kv4_scales4(uint32_t bytes, float (&s)[4]) {
    const uint32_t even = (bytes << 7) & 0x7f807f80u, odd = (bytes >> 1) & 0x7f807f80u;
    const float2 e = __half22float2(*reinterpret_cast<const __half2 *>(&even));
    const float2 o = __half22float2(*reinterpret_cast<const __half2 *>(&odd));
    s[0] = e.x;
    s[1] = o.x;
    s[2] = e.y;
    s[3] = o.y;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// cos and sin of pos * inv_freq as rope_cos_sin, in half turns (no slow path for large arguments).
__device__ __forceinline__ void kv4_cos_sin(int pos, double inv_freq, float &c, float &s) {
    const double kInvPi = 0.31830988618379067153776752674503;
    const double a = static_cast<double>(pos) * inv_freq * kInvPi;
    sincospif(static_cast<float>(a - 2.0 * rint(0.5 * a)), &s, &c);
}
__device__ __forceinline__ void kv4_rope4(float (&a)[4], int pos, const RopeFreqs &rf, int pairing, int lane) {
    if (pairing == kPairAdjacent) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float c, s;
            kv4_cos_sin(pos, rf.inv_freq[2 * lane + k], c, s);
            const float x = a[2 * k], y = a[2 * k + 1];
            a[2 * k] = x * c - y * s;
            a[2 * k + 1] = x * s + y * c;
        }
    } else {
        const float sign = lane < 16 ? -1.0f : 1.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float o = __shfl_xor_sync(0xffffffffu, a[k], 16);
            float c, s;
            kv4_cos_sin(pos, rf.inv_freq[4 * (lane & 15) + k], c, s);
            a[k] = fmaf(sign * o, s, a[k] * c);
        }
    }
}

constexpr int kKv4MinQuota = 8;       // least share of a team, in records
constexpr int kKv4PairCost = 24;      // what starting another pair costs, in records
constexpr int kKv4HeadPitch = 132;   // floats from one head's partial output in shared memory to the next

// Shape of kv4_decode_kernel for passes of HG query heads.  One CTA per SM, of teams of 4 warps; records that a warp takes
// at a time (two, for the instructions of the one to fill the waits of the other, where registers allow), times
// kStages in flight.
template <int HG>
struct Kv4Shape {
    static constexpr int kRecs = HG <= 8 ? 2 : 1;
    static constexpr int kStages = HG == 4 ? 2 : HG == 8 ? 3 : 4;
    static constexpr int kTeams = HG == 4 ? 4 : HG == 8 ? 3 : 2;
    static constexpr int kStageBytes = kRecs * kRec;
    static constexpr int kMerge = HG * kKv4HeadPitch * 4;
    static constexpr int kRing = (kStages * kStageBytes > kMerge ? kStages * kStageBytes : kMerge) + 127 & ~127;
    static constexpr int kSums = 32 * (HG == 16 ? 64 : 32);   // floats of a warp's O, for the long sums
    static constexpr int kBytes = kTeams * 4 * (kRing + kSums * 4);   // dynamic shared memory
    static constexpr int kQuantum = 4 * kRecs;          // a team's records are a multiple of this
};
constexpr int kKv4Sms = 148;
constexpr int kv4_teams(int HG) { return HG == 4 ? Kv4Shape<4>::kTeams : HG == 8 ? Kv4Shape<8>::kTeams : Kv4Shape<16>::kTeams; }

// Decode over a 4-bit cache.
//
//   S = q-hat K^T s_K / sqrt(D)      P = 2^(S - m)      O = sum P s_V c_V      (per warp, joined at the end)
//
// Work.  A pair is a (sequence, KV head, pass of HG query heads); it costs its records and kKv4PairCost for its
// prologue and epilogue.  The pairs' costs, one behind another, are dealt out in equal shares to the teams of all SMs, first
// the first teams', so lengths on the device decide and small work goes to all SMs.  (The teams of an SM are one CTA: as
// four CTAs with equal shares they ended after 154, 184, 216 and 245 us, since the older ones are favoured, as one after
// 218 to 222.)  A share begins and ends anywhere: a team goes through the segments of the pairs that it meets, and leaves
// (m, l, O) of each in slot pair + team (either moves on from one segment to the next, so slots are distinct); a
// pair within one team's share gets its output right away.  plan says where a pair's slots are.
// Within a segment every warp takes every fourth unit of one or two records.  Its lanes keep the bulk copies of the
// next units' records in flight, into the warp's own ring, so no warp waits for another before the segment's end.
// Both products are mma.m16n8k16 with the cache as the 16-row operand, S^T = K Q^T over 16 rows and
// O^T = V^T P^T over 16 elements, and the query heads as the 8 columns: a decode step has 1 to 16 query heads a KV head,
// so a tcgen05 tile of 128 rows of them would be at least 7/8 empty, and one of 128 cache rows would want fp16
// values in shared memory first (four times the bytes that were loaded).  q and P are split into two fp16
// numbers, 22 bits: up to 4 heads the two parts are neighbouring columns of one
// product, else a second product.  m moves only when a logit exceeds it by more than kMaxAhead; l and O are fp32.
// Bound by the latencies of what turns codes into fp16, which 16 warps an SM do not fill (65% of the issue slots used,
// 1.4 of 4 warps a scheduler ready), with the memory close behind: 64 sequences of 1K to 32K rows, 32/8 heads, take 230 us, 5.0
// TB/s; without the copies 212, without the products 182 (271 in a run long enough for the power cap to lower the clock).
// An append form (p.k_new): the warp that has the sequence's last record evaluates the new row while the records are
// on their way, and puts it into the cache and into its own copy of the record.
template <int HG, bool SCORES>
__global__ void __launch_bounds__(128 * Kv4Shape<HG>::kTeams, 1) kv4_decode_kernel(const __grid_constant__ Kv4DecodeParams p) {
    constexpr bool kPair = HG == 4;            // hi and lo of a head in neighbouring columns
    constexpr int kNT = HG == 16 ? 2 : 1;      // column tiles
    constexpr int kTerms = kPair ? 1 : 2;      // products a column tile
    constexpr int kLH = kPair ? 1 : 2 * kNT;   // query heads a lane holds logits of
    using Shape = Kv4Shape<HG>;
    constexpr int kR = Shape::kRecs, kStages = Shape::kStages, kBatch = 32 / kR;
    constexpr int kTeams = Shape::kTeams;
    extern __shared__ __align__(128) uint8_t s_all_rings[];   // [kTeams][4][kRing]
    __shared__ __align__(8) uint64_t s_all_bar[kTeams][4][kStages];
    __shared__ __align__(16) __half s_all_q[kTeams][2][HG][kHeadDim];
    __shared__ float s_all_f[kTeams][HG];
    __shared__ __align__(16) float s_all_new[kTeams][2][kHeadDim];   // the new row of k-hat and v
    __shared__ float s_all_m[kTeams][4][HG], s_all_l[kTeams][4][HG];
    __shared__ long long s_sum[4 * kTeams], s_off[kTeams];
    __shared__ int s_all_bad[kTeams], s_seq[kTeams];

    grid_dependency_wait();
    grid_dependents_launch();
    const int Hkv = p.cache.Hkv, P = Hkv * p.passes;   // pairs of a sequence
    const int team = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

    // ---- this team's share
    auto cost_of = [&](int b) {     // of a pair of sequence b: its records and kKv4PairCost
        int len;
        return kv4_seq_ok(p, b, len) ? (len + kRecRows - 1) / kRecRows + kKv4PairCost : 0;
    };
    const int self = team * gridDim.x + blockIdx.x;   // this team among all
    long long quota, pos, end;
    {
        constexpr int kT = 128 * kTeams;
        const int per = (p.B + kT - 1) / kT, b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
        long long sum = 0;
        for (int b = b0; b < b1; ++b) sum += cost_of(b);
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const int wid = threadIdx.x >> 5;
        if (lane == 31) s_sum[wid] = incl;
        __syncthreads();
        long long total = 0, before = incl - sum;
#pragma unroll
        for (int w = 0; w < 4 * kTeams; ++w) {
            if (w < wid) before += s_sum[w];
            total += s_sum[w];
        }
        total *= P;
        const unsigned teams = kTeams * gridDim.x;
        quota = ((total + teams - 1) / teams + Shape::kQuantum - 1) / Shape::kQuantum * Shape::kQuantum;
        if (quota < kKv4MinQuota) quota = kKv4MinQuota;
#pragma unroll
        for (int k = 0; k < kTeams; ++k) {   // where the share of each of this CTA's teams begins
            const long long at = (k * gridDim.x + blockIdx.x) * quota;
            if (at < total && before * P <= at && at < (before + sum) * P) {
                long long x = before * P;
                int b = b0;
                for (;; ++b) {
                    const long long n = static_cast<long long>(cost_of(b)) * P;
                    if (at < x + n) break;
                    x += n;
                }
                s_seq[k] = b;
                s_off[k] = at - x;
            }
        }
        __syncthreads();
        pos = self * quota;
        end = min(total, pos + quota);
        if (pos >= total) return;   // from here on teams go their own ways
    }
    auto sync_team = [&] { asm volatile("bar.sync %0, 128;" ::"r"(team + 1) : "memory"); };
    uint8_t *const s_rings = s_all_rings + team * 4 * Shape::kRing;
    auto &s_q = s_all_q[team];
    auto &s_f = s_all_f[team];
    auto &s_new = s_all_new[team];
    auto &s_m = s_all_m[team];
    auto &s_l = s_all_l[team];
    int &s_bad = s_all_bad[team];
    uint8_t *const my_ring = s_rings + warp * Shape::kRing;
    const uint32_t ring = smem_u32(my_ring), bars = smem_u32(s_all_bar[team][warp]);
    int b = s_seq[team], cost = cost_of(b);
    int sub = static_cast<int>(s_off[team] / cost), at = static_cast<int>(s_off[team] % cost);

    while (true) {
        // ---- one segment: records first .. first + nrec - 1 of the pair, where its cost is at .. till - 1
        const int till = static_cast<int>(min(static_cast<long long>(cost), at + (end - pos)));
        const int first = max(0, at - kKv4PairCost), nrec = max(0, till - kKv4PairCost) - first;
        const long long pair0 = pos - at;   // where the pair's cost begins
        pos += till - at;
        auto next_pair = [&] {   // there is one while pos < end: the last is not beyond it
            at = 0;
            if (++sub == P) {
                sub = 0;
                do cost = cost_of(++b);
                while (cost == 0);
            }
        };
        if (nrec == 0) {
            if (pos >= end) return;
            next_pair();
            continue;
        }
        const int kvh = sub / p.passes, jbase = sub % p.passes * HG;
        const int len = p.seqlens[b] + p.len_add;
        const bool last = till == cost, whole = last && first == 0;
        const long long pair = static_cast<long long>(b) * P + sub;
        const int units = (nrec + kR - 1) / kR;
        const int todo = units > warp ? (units - warp + 3) >> 2 : 0;   // units warp, warp + 4, ...
        const int rows_end = min(len, (first + nrec) * kRecRows);
        if (tid == 0) {
            s_bad = 0;
            if (first == 0)
                p.plan[pair] = make_int2(self, static_cast<int>((pair0 + cost - 1) / quota) - self + 1);
        }

        // lane l finds record l % kR of the warp's unit kBatch n + l / kR.  A page out of range: any record in its
        // place, and the result is poisoned.
        bool bad = false;
        auto row_of = [&](int i) { return (first + (4 * i + warp) * kR + lane % kR) * kRecRows; };
        auto page_of = [&](int i) {   // the table's entry, looked at later
            return i < todo && row_of(i) < rows_end
                       ? p.cache.table[static_cast<size_t>(b) * p.cache.max_pages + row_of(i) / p.cache.page_size]
                       : 0;
        };
        auto locate = [&](int i, int page) -> const uint8_t * {
            if (i >= todo || row_of(i) >= rows_end) return nullptr;
            const bool ok = page >= 0 && page < p.cache.num_pages;
            bad |= !ok;
            return ok ? kv4_record(p.cache, page, kvh, row_of(i) % p.cache.page_size) : p.cache.recs;
        };
        const int page0 = page_of(lane / kR);
        int next_page = page_of(kBatch + lane / kR);
        const int ps = p.qpos ? p.qpos[b] : p.seqlens[b];
        uint2 raw[HG / 4];   // q of heads warp, warp + 4, ...: on its way with the table's entries
#pragma unroll
        for (int x = 0; x < HG / 4; ++x)
            if (jbase + warp + 4 * x < p.hpg)
                raw[x] = *reinterpret_cast<const uint2 *>(
                    p.q + (static_cast<size_t>(b) * p.H + kvh * p.hpg + jbase + warp + 4 * x) * kHeadDim + 4 * lane);
        const uint8_t *my_rec = locate(lane / kR, page0);
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, kR);
            fence_mbarrier_init();
            fence_proxy_async_smem();
        }
        __syncwarp();
        auto request = [&](int st) {   // the copy of this lane's record into stage st
            if (my_rec == nullptr) {
                mbar_arrive(bars + 8 * st);
                return;
            }
            mbar_arrive_expect_tx(bars + 8 * st, kRec);
            bulk_load(ring + st * Shape::kStageBytes + lane % kR * kRec, my_rec, kRec, bars + 8 * st);
        };
#pragma unroll
        for (int st = 0; st < kStages; ++st)
            if (st < todo && lane / kR == st) request(st);

        // ---- q prologue: RMSNorm + RoPE, and by a power of two per head into fp16's range
        {
            const float4 w = reinterpret_cast<const float4 *>(p.wq)[lane];
#pragma unroll
            for (int x = 0; x < HG / 4; ++x) {
                const int j = warp + 4 * x;
                float y[4] = {0.f, 0.f, 0.f, 0.f};
                if (jbase + j < p.hpg) {
                    const float x0 = bf16lo(raw[x].x), x1 = bf16hi(raw[x].x), x2 = bf16lo(raw[x].y), x3 = bf16hi(raw[x].y);
                    float ss = x0 * x0 + x1 * x1 + x2 * x2 + x3 * x3;
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float inv = 1.0f / sqrtf(ss * (1.0f / kHeadDim) + p.eps);
                    y[0] = w.x * x0 * inv;
                    y[1] = w.y * x1 * inv;
                    y[2] = w.z * x2 * inv;
                    y[3] = w.w * x3 * inv;
                    kv4_rope4(y, ps, p.rf, p.pairing, lane);   // warp-uniform: j depends on the warp only
                }
                float am = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
                const int e = max(static_cast<int>(__float_as_uint(am) >> 23) - 127, -100);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);   // largest magnitude in [2^14, 2^15)
                uint32_t h0, l0, h1, l1;
                h2_split(y[0] * up, y[1] * up, h0, l0);
                h2_split(y[2] * up, y[3] * up, h1, l1);
                *reinterpret_cast<uint2 *>(&s_q[0][j][4 * lane]) = make_uint2(h0, h1);
                *reinterpret_cast<uint2 *>(&s_q[1][j][4 * lane]) = make_uint2(l0, l1);
                if (lane == 0) s_f[j] = __uint_as_float(static_cast<uint32_t>(127 + e - 14) << 23) * p.scale_log2;
            }
        }
        sync_team();

        // ---- the new row
        // the warp's last unit, where rows of it lie behind the segment or the new one is among them
        const bool owns_new = last && p.k_new != nullptr && warp == ((units - 1) & 3);
        const int special = owns_new || (first + (4 * (todo - 1) + warp + 1) * kR) * kRecRows > rows_end ? todo - 1 : -1;
        if (owns_new) {
            float kn[4], vn[4];
            kv4_new_row(p, b, kvh, kn, vn, lane);
            reinterpret_cast<float4 *>(s_new[0])[lane] = make_float4(kn[0], kn[1], kn[2], kn[3]);
            reinterpret_cast<float4 *>(s_new[1])[lane] = make_float4(vn[0], vn[1], vn[2], vn[3]);
            const int page = kv4_page(p.cache, b, len - 1);
            if (jbase == 0 && page >= 0)
                kv4_store_row(kv4_record(p.cache, page, kvh, (len - 1) % p.cache.page_size), (len - 1) % kRecRows, kn, vn, lane);
            __syncwarp();
        }

        // B fragments of q: elements 16 s + 4 t .. + 3 of column g
        uint2 qb[kNT][kTerms][8];
        float f[kLH];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int u = 0; u < kTerms; ++u)
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    qb[nt][u][s] = *reinterpret_cast<const uint2 *>(
                        kPair ? &s_q[g & 1][g >> 1][16 * s + 4 * t] : &s_q[u][(8 * nt + g) % HG][16 * s + 4 * t]);
        auto head = [&](int x) { return kPair ? t : 8 * (x >> 1) + 2 * t + (x & 1); };   // of the lane's logits x
#pragma unroll
        for (int x = 0; x < kLH; ++x) f[x] = s_f[head(x)] * kCodeUnit;

        const uint32_t base0 = p.base0, base1 = p.base1;
        float o[kNT][8][4];   // [tile T]: elements 16 g + 2 T (0, 1) and + 1 (2, 3) of columns 2 t, 2 t + 1
        float m[kLH], l[kLH];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
#pragma unroll
        for (int x = 0; x < kLH; ++x) {
            m[x] = -INFINITY;
            l[x] = 0.f;
        }

        // The matrix instruction cuts off what does not fit into its fp32 sums (it does not round), so a long sum of
        // like terms would come out small: every kBatch units O is added to sums in shared memory, as of maximum m_sums, and l
        // to l_sums (as one long sum l would round off small weights beside a large one that O holds).
        float4 *const sums = reinterpret_cast<float4 *>(s_all_rings + kTeams * 4 * Shape::kRing) +
                             (team * 4 + warp) * (Shape::kSums / 4) + lane;
        float m_sums[kLH], l_sums[kLH];
        auto collect = [&](bool any) {   // o += the sums so far
            if (!any) return;
            float r[kLH];
#pragma unroll
            for (int x = 0; x < kLH; ++x) {
                r[x] = ex2_approx(m_sums[x] - m[x]);
                l[x] = fmaf(l_sums[x], r[x], l[x]);
            }
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float4 v = sums[(8 * nt + n) * 32];
                    const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][n][e] = fmaf(y[e], r[kPair ? 0 : 2 * nt + (e & 1)], o[nt][n][e]);
                }
        };
#pragma unroll 1
        for (int i = 0, st = 0, parity = 0; i < todo; ++i) {
            if (((i + kStages) & (kBatch - 1)) == 0) {
                my_rec = locate(i + kStages + lane / kR, next_page);
                next_page = page_of(i + kStages + kBatch + lane / kR);
                if (i > 0) {   // at most 64 products go into an accumulator before it is added up here
                    collect(i > kBatch);
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            sums[(8 * nt + n) * 32] = make_float4(o[nt][n][0], o[nt][n][1], o[nt][n][2], o[nt][n][3]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt][n][e] = 0.f;
                        }
#pragma unroll
                    for (int x = 0; x < kLH; ++x) {
                        m_sums[x] = m[x];
                        l_sums[x] = l[x];
                        l[x] = 0.f;
                    }
                }
            }
            if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * st, parity, p.err))) {
                // the copies in flight land before their shared memory is used again
                for (int j = i; j < min(todo, i + kStages); ++j)
                    mbar_wait(bars + 8 * (j % kStages), (j / kStages) & 1, p.err);
                bad = true;
                break;
            }
            uint8_t *unit = my_ring + st * Shape::kStageBytes;
            const int row0 = (first + (4 * i + warp) * kR) * kRecRows;
            if (i == special) {
                if (owns_new) {
                    const float4 k4 = reinterpret_cast<const float4 *>(s_new[0])[lane];
                    const float4 v4 = reinterpret_cast<const float4 *>(s_new[1])[lane];
                    const float kn[4] = {k4.x, k4.y, k4.z, k4.w}, vn[4] = {v4.x, v4.y, v4.z, v4.w};
                    kv4_store_row(unit + (len - 1 - row0) / kRecRows * kRec, (len - 1) % kRecRows, kn, vn, lane);
                }
                if (lane < kR * kRecRows && row0 + lane >= rows_end)   // they weigh nothing, whatever their bytes
#pragma unroll
                    for (int e = 0; e < 4; ++e) unit[lane / kRecRows * kRec + kRecVs + 16 * e + lane % kRecRows] = 0;
                __syncwarp();
            }
            // ---- logits (without their factor f > 0): lane (g, t) gets rows g and g + 8 of each record, of columns 2 t, 2 t + 1
            float lg[kLH][2 * kR];
#pragma unroll
            for (int h = 0; h < kR; ++h) {
                const uint8_t *rec = unit + h * kRec;
                const uint4 ka = *reinterpret_cast<const uint4 *>(rec + 16 * lane);
                const uint4 kb = *reinterpret_cast<const uint4 *>(rec + 512 + 16 * lane);
                float sa[4], sb[4];
                kv4_scales4(*reinterpret_cast<const uint32_t *>(rec + kRecKs + 4 * g), sa);
                kv4_scales4(*reinterpret_cast<const uint32_t *>(rec + kRecKs + 32 + 4 * g), sb);
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int x = 0; x < kLH; ++x) lg[x][2 * h] = lg[x][2 * h + 1] = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint32_t ya = wa[w] >> (8 * u), yb = wb[w] >> (8 * u);
                            const uint32_t a0 = h2_add(kv4_pick<kCodeMask0>(ya, base0), kCodeOff0);
                            const uint32_t a1 = h2_add(kv4_pick<kCodeMask0>(yb, base0), kCodeOff0);
                            const uint32_t a2 = h2_add(kv4_pick<kCodeMask1>(ya, base1), kCodeOff1);
                            const uint32_t a3 = h2_add(kv4_pick<kCodeMask1>(yb, base1), kCodeOff1);
#pragma unroll
                            for (int term = 0; term < kTerms; ++term) {
                                const uint2 q2 = qb[nt][term][2 * w + u];
                                mma16816(c, a0, a1, a2, a3, q2.x, q2.y);
                            }
                        }
                        if constexpr (kPair) {
                            lg[0][2 * h] = fmaf(c[0] + c[1], sa[w], lg[0][2 * h]);
                            lg[0][2 * h + 1] = fmaf(c[2] + c[3], sb[w], lg[0][2 * h + 1]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int x = 2 * nt + e;
                                lg[x][2 * h] = fmaf(c[e], sa[w], lg[x][2 * h]);
                                lg[x][2 * h + 1] = fmaf(c[2 + e], sb[w], lg[x][2 * h + 1]);
                            }
                        }
                    }
                }
            }
            if (i == special) {
#pragma unroll
                for (int x = 0; x < kLH; ++x)
#pragma unroll
                    for (int r = 0; r < 2 * kR; ++r)
                        if (row0 + g + 8 * r >= rows_end) lg[x][r] = -INFINITY;
            }
            if constexpr (SCORES) {
#pragma unroll
                for (int x = 0; x < kLH; ++x)
                    if (jbase + head(x) < p.hpg) {
                        float *dst = p.scores + (static_cast<size_t>(b) * p.H + kvh * p.hpg + jbase + head(x)) * p.score_stride + row0 + g;
#pragma unroll
                        for (int r = 0; r < 2 * kR; ++r)
                            if (row0 + g + 8 * r < rows_end) dst[8 * r] = lg[x][r] * f[x];
                    }
            }
            // ---- running maximum and sum
            bool move = false;
            float top[kLH];
#pragma unroll
            for (int x = 0; x < kLH; ++x) {
                top[x] = fmaxf(lg[x][0], lg[x][1]);
#pragma unroll
                for (int r = 2; r < 2 * kR; ++r) top[x] = fmaxf(top[x], lg[x][r]);
                top[x] *= f[x];
                move |= top[x] > m[x] + kMaxAhead;
            }
            if (__any_sync(0xffffffffu, move)) {
                float r[kLH];
#pragma unroll
                for (int x = 0; x < kLH; ++x) {
                    float mx = top[x];
#pragma unroll
                    for (int s = 4; s <= 16; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                    const float mn = fmaxf(m[x], mx);
                    r[x] = ex2_approx(m[x] - mn);
                    m[x] = mn;
                    l[x] *= r[x];
                }
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[nt][n][e] *= r[kPair ? 0 : 2 * nt + (e & 1)];
            }
#pragma unroll
            for (int x = 0; x < kLH; ++x) {
                float sum = 0.f;
#pragma unroll
                for (int r = 0; r < 2 * kR; ++r) {
                    lg[x][r] = ex2_approx(fmaf(lg[x][r], f[x], -m[x]));
                    sum += lg[x][r];
                }
                l[x] += sum;
            }
#pragma unroll
            for (int h = 0; h < kR; ++h) {
                // B fragments of P: rows 2 t, 2 t + 1 (and + 8) of column g
                uint32_t pb[kNT][kTerms][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if constexpr (kPair) {
                        const float pr = lg[0][2 * h + e] * kWeightUnit, rest = pr - __half2float(__float2half_rn(pr));
                        uint32_t both;
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(both) : "f"(rest), "f"(pr));
                        pb[0][0][e] = transpose8x8(both);
                    } else {
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            uint32_t hi, lo;
                            h2_split(lg[2 * nt][2 * h + e] * kWeightUnit, lg[2 * nt + 1][2 * h + e] * kWeightUnit, hi, lo);
                            pb[nt][0][e] = transpose8x8(hi);
                            pb[nt][kTerms - 1][e] = transpose8x8(lo);
                        }
                    }
                }
                // ---- O^T += V^T P^T: lane (g, t) feeds rows 2t, 2t + 1, 8 + 2t, 8 + 2t + 1 of elements 16 g ..
                const uint8_t *rec = unit + h * kRec;
                const uint4 va = *reinterpret_cast<const uint4 *>(rec + kRecV + 16 * lane);
                const uint4 vb = *reinterpret_cast<const uint4 *>(rec + kRecV + 512 + 16 * lane);
                const uint8_t *vs = rec + kRecVs + 16 * (g >> 1) + 2 * t;
                const Kv4Scale2 s0 = kv4_scale2(*reinterpret_cast<const uint16_t *>(vs));
                const Kv4Scale2 s1 = kv4_scale2(*reinterpret_cast<const uint16_t *>(vs + 8));
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t sel = u ? 0x7632u : 0x5410u;   // the same half word of two rows
                        const uint32_t xa = __byte_perm(w ? va.y : va.x, w ? va.w : va.z, sel);
                        const uint32_t xb = __byte_perm(w ? vb.y : vb.x, w ? vb.w : vb.z, sel);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t ya = xa >> (8 * j), yb = xb >> (8 * j);
                            const uint32_t a0 = h2_fma(kv4_pick<kCodeMask0>(ya, base0), s0.s, s0.o0), a1 = h2_fma(kv4_pick<kCodeMask1>(ya, base1), s0.s, s0.o1);
                            const uint32_t a2 = h2_fma(kv4_pick<kCodeMask0>(yb, base0), s1.s, s1.o0), a3 = h2_fma(kv4_pick<kCodeMask1>(yb, base1), s1.s, s1.o1);
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                                for (int term = 0; term < kTerms; ++term)
                                    mma16816(o[nt][4 * w + 2 * u + j], a0, a1, a2, a3, pb[nt][term][0], pb[nt][term][1]);
                        }
                    }
            }
            __syncwarp();
            if (lane / kR == ((i + kStages) & (kBatch - 1)) && i + kStages < todo) request(st);
            if (++st == kStages) {
                st = 0;
                parity ^= 1;
            }
        }
        collect(todo > kBatch - kStages);   // there are some from unit kBatch - kStages on
        if (bad) s_bad = 1;

        // ---- join the four warps: lane (g, t) holds elements 16 g .. 16 g + 15 of its heads
        float *so = reinterpret_cast<float *>(my_ring);
#pragma unroll
        for (int x = 0; x < kLH; ++x) {
            float *dst = so + head(x) * kKv4HeadPitch + 16 * g;
            const int nt = x >> 1, c = x & 1;
#pragma unroll
            for (int n = 0; n < 8; n += 2) {
                if constexpr (kPair)
                    *reinterpret_cast<float4 *>(dst + 2 * n) =
                        make_float4(o[0][n][0] + o[0][n][1], o[0][n][2] + o[0][n][3], o[0][n + 1][0] + o[0][n + 1][1],
                                    o[0][n + 1][2] + o[0][n + 1][3]);
                else
                    *reinterpret_cast<float4 *>(dst + 2 * n) =
                        make_float4(o[nt][n][c], o[nt][n][2 + c], o[nt][n + 1][c], o[nt][n + 1][2 + c]);
            }
#pragma unroll
            for (int s = 4; s <= 16; s <<= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], s);
            if (g == 0) {
                s_m[warp][head(x)] = m[x];
                s_l[warp][head(x)] = l[x];
            }
        }
        sync_team();
        const bool poison = s_bad != 0;
        if (poison && tid == 0) atomicOr(p.err, kErrInput);
        const size_t slot = static_cast<size_t>(pair + self) * HG;
#pragma unroll 1
        for (int j = 0; j < HG && jbase + j < p.hpg; ++j) {
            float M = s_m[0][j];
#pragma unroll
            for (int w = 1; w < 4; ++w) M = fmaxf(M, s_m[w][j]);
            float O = 0.f, L = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float r = ex2_approx(s_m[w][j] - M);
                O = fmaf(r, reinterpret_cast<const float *>(s_rings + w * Shape::kRing)[j * kKv4HeadPitch + tid], O);
                L = fmaf(r, s_l[w][j], L);
            }
            O *= kCodeUnit / kWeightUnit;
            if (poison) {
                O = L = __int_as_float(0x7fc00000);
                M = 0.f;
            }
            if (whole)
                p.out[(static_cast<size_t>(b) * p.H + kvh * p.hpg + jbase + j) * kHeadDim + tid] = O / L;
            else
                p.part_o[(slot + j) * kHeadDim + tid] = O;
            if (tid == 0 && (SCORES || !whole)) {
                p.part_ml[2 * (slot + j)] = M;
                p.part_ml[2 * (slot + j) + 1] = L;
            }
        }
        if (pos >= end) return;
        next_pair();
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < kStages; ++i) mbar_inval(bars + 8 * i);
        fence_proxy_async_smem();   // the ring goes back to the copies
        sync_team();
    }
}

}  // namespace gqa
