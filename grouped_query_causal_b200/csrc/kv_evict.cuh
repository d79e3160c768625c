// kv_evict.cuh -- the attention weight that every cached row receives, accumulated over decode steps, and eviction
// of a cache down to a budget of rows by that weight.
//
//  decode_finish_kernel: joins the chunks of a decode step, and weights[b][g][r] += sum over the query heads of
//                     group g of 2^(S[r] - M) / L, from the logits S that the decode kernels leave in the
//                     workspace and the joined M and L of every head.
//  kv_select_kernel:  which rows stay (one CTA per sequence and KV head, or a cluster of up to 8 that share the rows): the
//                     `budget` rows of the greatest key, ties to the lowest row, by a radix selection over 32-bit keys.
//  kv_move_kernel:    the rows themselves.  Keys are rotated before they are cached, so a sequence's rows have no
//                     order that attention would see: kept rows below the budget stay where they are, and the i-th kept
//                     row behind it goes to the i-th free row below it.  Sources lie behind the budget and targets
//                     below it, so the moves run in place and in any order, and no row moves that need not.
#pragma once
#include <climits>
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "ptx.cuh"

namespace gqa {

// The cached rows of a batch: contiguous (offsets) or paged (pages).
struct SeqRows {
    const int64_t *offsets;   // [B + 1] or nullptr
    const int32_t *seqlens;   // [B]
    const int32_t *pages;     // [B, max_pages] or nullptr
    int page_size, max_pages, num_pages;
    int max_len, len_add;
};

// len = seqlens[b] + len_add rows, at least `least` of them, within the bound and the sequence's rows.
__device__ __forceinline__ bool seq_rows_ok(const SeqRows &s, int b, int least, int &len) {
    len = s.seqlens[b] + s.len_add;
    long long cap;
    if (s.pages != nullptr) {
        cap = static_cast<long long>(s.max_pages) * s.page_size;
    } else {
        if (s.offsets[b] < 0) return false;
        cap = s.offsets[b + 1] - s.offsets[b];
    }
    return len >= least && len <= s.max_len && static_cast<long long>(len) <= cap;
}

// ------------------------------------------------------------------ joining the chunks, accumulation
struct FinishParams {
    SeqRows rows;
    const int32_t *qpos;      // [B] or nullptr
    const float *part_o;      // [slots, D]
    const float *part_ml;     // [slots, 2]
    const int2 *plan;         // kv4_decode_kernel's, or nullptr: decode_split_kernel's chunks
    const float *scores;      // [B * H, score_stride]
    long long score_stride;
    float *out;               // [B, H, D]
    float *weights;           // [B, Hkv, wstride]
    int32_t *row_pos;         // [B, Hkv, wstride] or nullptr
    long long wstride;
    unsigned *err;
    int H, Hkv, hpg;
    int group;                // with a plan: query heads of a pass
    int maxC, chunk;          // without one
    int tile;                 // rows a CTA accumulates, a multiple of kAccRows
};

constexpr int kAccRows = 1024;   // rows a CTA accumulates at a time
constexpr int kAccHeads = 64;    // query heads whose M and 1 / L are held at a time

// Where the parts of query head j of (sequence b, KV head g) are: slots first, first + step, ...
struct FinishSlots {
    size_t first;
    int step, n;
};
__device__ __forceinline__ FinishSlots finish_slots(const FinishParams &p, int b, int g, int j, int len) {
    FinishSlots s;
    if (p.plan != nullptr) {
        const int passes = (p.hpg + p.group - 1) / p.group;
        const size_t pair = (static_cast<size_t>(b) * p.Hkv + g) * passes + j / p.group;
        const int2 at = p.plan[pair];
        s.first = (pair + at.x) * p.group + j % p.group;
        s.step = p.group;
        s.n = at.y;
    } else {
        s.first = static_cast<size_t>(b) * p.maxC * p.H + static_cast<size_t>(g) * p.hpg + j;
        s.step = p.H;
        s.n = (len + p.chunk - 1) / p.chunk;
    }
    return s;
}

// The joined maximum and sum of one query head, by one warp.
__device__ __forceinline__ float2 finish_stats(const FinishParams &p, const FinishSlots &s, int lane) {
    float M = -INFINITY, L = 0.f;
    for (int c = lane; c < s.n; c += 32) M = fmaxf(M, p.part_ml[2 * (s.first + static_cast<size_t>(c) * s.step)]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int c = lane; c < s.n; c += 32) {
        const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + 2 * (s.first + static_cast<size_t>(c) * s.step));
        L = fmaf(ex2_approx(ml.x - M), ml.y, L);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    return make_float2(M, L);
}

// After the parts of a decode step: out = sum_c 2^(m_c - M) O_c / L for every query head, and with ACC the
// weights of the rows.  256 threads a CTA; of the gridDim.y CTAs of a (sequence, KV head) the first `tiles` accumulate
// p.tile rows each, the others join a head each.  Bound by memory: 512 B a part and head, 4 B a logit, 8 B a weight; loads
// that do not depend on one another are issued together, since a CTA lives for a few of their latencies only.  The
// parts of decode_split_kernel are summed as decode_merge_kernel does, for the same bits; those of
// kv4_decode_kernel, of which one sequence may have hundreds, and smaller chunks by eight warps at once.  A step whose softmax is not a
// number (a bad page, a NaN in the cache) leaves the weights as they were.
template <bool ACC>
__global__ void __launch_bounds__(256) decode_finish_kernel(const __grid_constant__ FinishParams p) {
    __shared__ __align__(16) float s_o[8][kHeadDim];
    __shared__ float2 s_ml[kAccHeads];
    __shared__ int s_nan;
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles = ACC ? (p.rows.max_len + p.tile - 1) / p.tile : 0;
    int len;
    const bool ok = seq_rows_ok(p.rows, b, 1, len);
    const size_t head0 = static_cast<size_t>(b) * p.H + static_cast<size_t>(g) * p.hpg;
    if (static_cast<int>(blockIdx.y) >= tiles) {
        for (int j = blockIdx.y - tiles; j < p.hpg; j += gridDim.y - tiles) {
            float *out = p.out + (head0 + j) * kHeadDim;
            if (!ok) {
                if (tid < kHeadDim) out[tid] = __int_as_float(0x7fc00000);
                if (tid == 0 && g == 0 && j == 0) atomicOr(p.err, kErrInput);
                continue;
            }
            const FinishSlots s = finish_slots(p, b, g, j, len);
            if (p.plan == nullptr && p.chunk == kChunk) {
                if (tid >= kHeadDim) continue;
                float M = -INFINITY, O = 0.f, L = 0.f;
#pragma unroll 8
                for (int c = 0; c < s.n; ++c) M = fmaxf(M, p.part_ml[2 * (s.first + static_cast<size_t>(c) * s.step)]);
#pragma unroll 8
                for (int c = 0; c < s.n; ++c) {
                    const size_t slot = s.first + static_cast<size_t>(c) * s.step;
                    const float r = ex2_approx(p.part_ml[2 * slot] - M);
                    O = fmaf(r, p.part_o[slot * kHeadDim + tid], O);
                    L = fmaf(r, p.part_ml[2 * slot + 1], L);
                }
                out[tid] = O / L;
                continue;
            }
            if (p.plan != nullptr && s.n == 1) continue;   // written already
            constexpr int kAhead = 4;
            float4 x[kAhead];
            float m[kAhead];
            auto load = [&](int c0) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int c = c0 + 8 * i;
                    const size_t slot = s.first + static_cast<size_t>(c) * s.step;
                    x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    m[i] = -INFINITY;
                    if (c < s.n) {
                        x[i] = reinterpret_cast<const float4 *>(p.part_o + slot * kHeadDim)[lane];
                        m[i] = p.part_ml[2 * slot];
                    }
                }
            };
            load(warp);
            const float2 ml = finish_stats(p, s, lane);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c0 = warp; c0 < s.n; c0 += 8 * kAhead) {
                if (c0 != warp) load(c0);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (c0 + 8 * i >= s.n) continue;
                    const float r = ex2_approx(m[i] - ml.x);
                    o.x = fmaf(r, x[i].x, o.x);
                    o.y = fmaf(r, x[i].y, o.y);
                    o.z = fmaf(r, x[i].z, o.z);
                    o.w = fmaf(r, x[i].w, o.w);
                }
            }
            __syncthreads();
            reinterpret_cast<float4 *>(s_o[warp])[lane] = o;
            __syncthreads();
            if (tid < kHeadDim) {
                float O = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) O += s_o[w][tid];
                out[tid] = O / ml.y;
            }
        }
        return;
    }
    if constexpr (ACC) {
        const int begin = blockIdx.y * p.tile, end = min(len, begin + p.tile);
        if (!ok || begin >= end) return;
        constexpr int kHeads = 4;
        bool bad = false;
        for (int r0 = begin; r0 < end; r0 += kAccRows) {
            const float *s = p.scores + head0 * p.score_stride + r0 + tid;
            const size_t base = (static_cast<size_t>(b) * p.Hkv + g) * p.wstride + r0 + tid;
            float x[kHeads][4], w[4], old[4];
            bool in[4];
            auto load = [&](int j0) {
#pragma unroll
                for (int j = 0; j < kHeads; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[j][i] = in[i] && j0 + j < p.hpg ? s[(j0 + j) * p.score_stride + 256 * i] : -INFINITY;
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + tid + 256 * i;
                in[i] = r < end;
                w[i] = 0.f;
                old[i] = in[i] && !(p.rows.len_add && r == len - 1) ? p.weights[base + 256 * i] : 0.f;   // an appended row starts from zero
            }
            load(0);
            for (int j0 = 0; j0 < p.hpg && !bad; j0 += kAccHeads) {
                const int nj = min(kAccHeads, p.hpg - j0);
                if (r0 == begin || p.hpg > kAccHeads) {   // else they are there
                    __syncthreads();
                    if (tid == 0) s_nan = 0;
                    __syncthreads();
                    for (int j = warp; j < nj; j += 8) {
                        const float2 ml = finish_stats(p, finish_slots(p, b, g, j0 + j, len), lane);
                        if (lane == 0) {
                            s_ml[j] = make_float2(ml.x, 1.0f / ml.y);
                            if (!(ml.y > 0.f && ml.y < INFINITY)) s_nan = 1;
                        }
                    }
                    __syncthreads();
                    bad = s_nan != 0;
                    if (bad) break;
                }
                for (int j = 0; j < nj; j += kHeads) {
                    if (j0 + j != 0) load(j0 + j);
#pragma unroll
                    for (int y = 0; y < kHeads; ++y) {
                        if (j + y >= nj) break;
                        const float2 ml = s_ml[j + y];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = fmaf(ex2_approx(x[y][i] - ml.x), ml.y, w[i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + tid + 256 * i;
                if (!in[i]) continue;
                const bool added = p.rows.len_add && r == len - 1;
                if (!bad || added) p.weights[base + 256 * i] = bad ? 0.f : old[i] + w[i];
                if (added && p.row_pos) p.row_pos[base + 256 * i] = p.qpos ? p.qpos[b] : r;
            }
        }
    }
}

// ------------------------------------------------------------------ selection
enum { kEvictRows = 0, kEvictPages = 1, kEvictKv4 = 2 };

struct KvEvictParams {
    SeqRows rows;
    uint16_t *k, *v;          // bf16 caches (kEvictRows, kEvictPages)
    Kv4Cache c4;              // kEvictKv4
    const float *weights;     // [B, Hkv, wstride]
    const int32_t *row_pos;   // [B, Hkv, wstride] or nullptr
    long long wstride;
    float *new_weights;       // [B, Hkv, new_wstride]; may be the same buffers
    int32_t *new_row_pos;
    long long new_wstride;
    int32_t *new_seqlens;     // [B]
    int32_t *moves;           // [B * Hkv][2][move_cap]: sources, then targets
    int32_t *counts;          // [B * Hkv]
    unsigned *err;
    int Hkv, budget, recent, move_cap;
    int key_cap, pos_cap;     // rows whose keys and positions fit into shared memory
    int cluster;              // CTAs of a (sequence, KV head)
    int copy;                 // the new metadata are other buffers: rows that stay are copied
    int fused;                // the selecting CTA moves the rows itself
};

// Row r (< 2^31) of sequence b as an index into rows of Hkv heads.
__device__ __forceinline__ long long evict_row(const KvEvictParams &p, int b, int r) {
    if (p.rows.pages == nullptr) return p.rows.offsets[b] + r;
    const int id = p.rows.pages[static_cast<size_t>(b) * p.rows.max_pages + r / p.rows.page_size];
    return static_cast<long long>(id) * p.rows.page_size + r % p.rows.page_size;
}

// Moves `first`, `first + step`, ... of one (sequence, KV head) by one warp, four rows (4-bit: eight) at a time
// so that their loads are in flight together.
template <int KIND>
__device__ __forceinline__ void evict_move(const KvEvictParams &p, int b, int g, const int32_t *src, const int32_t *dst,
                                           int n, int first, int step, int lane) {
    constexpr int kPer = KIND == kEvictKv4 ? 2 : 1;   // rows per warp access
    constexpr int kDeep = 4;
    const int sub = KIND == kEvictKv4 ? lane >> 4 : 0;
    const int h = lane & 15;
    for (int i0 = first * kPer * kDeep; i0 < n; i0 += step * kPer * kDeep) {
        uint4 x[kDeep];
        uint32_t sc[kDeep];
        int to[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            const int i = i0 + u * kPer + sub;
            to[u] = -1;
            if (i >= n) continue;
            const int from = src[i];
            to[u] = dst[i];
            if constexpr (KIND == kEvictKv4) {
                const int id = p.c4.table[static_cast<size_t>(b) * p.c4.max_pages + from / p.c4.page_size];
                const uint8_t *rec = kv4_record(p.c4, id, g, from % p.c4.page_size);
                const int r = from % kRecRows;
                const uint8_t *at = h < 8 ? rec + 64 * r + 8 * h
                                          : rec + kRecV + 512 * (r >> 3) + 64 * (h - 8) + 16 * ((r & 7) >> 1) + 8 * (r & 1);
                const uint2 y = *reinterpret_cast<const uint2 *>(at);
                x[u].x = y.x;
                x[u].y = y.y;
                if (h < 4) sc[u] = rec[kRecVs + 16 * h + r];
                if (h == 4) sc[u] = *reinterpret_cast<const uint32_t *>(rec + kRecKs + 4 * r);
            } else {
                const uint16_t *base = lane < 16 ? p.k : p.v;
                x[u] = *reinterpret_cast<const uint4 *>(base + (static_cast<size_t>(evict_row(p, b, from)) * p.Hkv + g) * kHeadDim + 8 * h);
            }
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            if (to[u] < 0) continue;
            if constexpr (KIND == kEvictKv4) {
                const int id = p.c4.table[static_cast<size_t>(b) * p.c4.max_pages + to[u] / p.c4.page_size];
                uint8_t *rec = kv4_record(p.c4, id, g, to[u] % p.c4.page_size);
                const int r = to[u] % kRecRows;
                uint8_t *at = h < 8 ? rec + 64 * r + 8 * h
                                    : rec + kRecV + 512 * (r >> 3) + 64 * (h - 8) + 16 * ((r & 7) >> 1) + 8 * (r & 1);
                *reinterpret_cast<uint2 *>(at) = make_uint2(x[u].x, x[u].y);
                if (h < 4) rec[kRecVs + 16 * h + r] = static_cast<uint8_t>(sc[u]);
                if (h == 4) *reinterpret_cast<uint32_t *>(rec + kRecKs + 4 * r) = sc[u];
            } else {
                uint16_t *base = lane < 16 ? p.k : p.v;
                *reinterpret_cast<uint4 *>(base + (static_cast<size_t>(evict_row(p, b, to[u])) * p.Hkv + g) * kHeadDim + 8 * h) = x[u];
            }
        }
    }
}

// The order of the weights as unsigned numbers: by value, NaN above infinity; the recent rows above all.
__device__ __forceinline__ uint32_t evict_key(float w, bool recent) {
    if (recent) return 0xffffffffu;
    if (isnan(w)) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(w + 0.0f);   // -0 counts as 0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

constexpr int kSelBins = 2048;
constexpr int kSelBytes = 192 * 1024;   // of shared memory for keys and positions
constexpr int kSelList = 1024;          // keys of one bin that are looked at by themselves
constexpr int kSelRank = 128;           // ... by comparing each with each

// Sum of `x` over the threads before this one, and over all of them (s: 33 ints, free again after the next barrier).
__device__ __forceinline__ int block_scan(int x, int *s, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) s[warp] = incl;
    __syncthreads();
    int v = lane < warps ? s[lane] : 0;
    total = __reduce_add_sync(0xffffffffu, v);
    v = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
    return v + incl - x;
}

// A cluster of p.cluster CTAs (one where there are many pairs) per (sequence, KV head), each with a part of the rows.
// Weights and positions are read once, into shared memory (rows beyond key_cap and pos_cap are read again).  A
// histogram of the keys' upper 11 bits finds the bin of the budget-th greatest; the few keys of that bin are collected and
// compared with one another, more of them go through two more histograms, and where there are too many to collect all
// rows do.  Then every thread goes through consecutive rows (an odd number,
// so that shared memory has no conflicts), and scans over the threads give each its place among the ties, the holes below the
// budget and the kept rows behind it, in order of rows.  Bound by the latency of its barriers where rows are few, else by
// an SM's reads and shared-memory atomics.
template <int KIND>
__global__ void __launch_bounds__(1024) kv_select_kernel(const __grid_constant__ KvEvictParams p) {
    extern __shared__ uint32_t s_key[];   // [key_cap], then positions [pos_cap]
    __shared__ __align__(16) int s_hist[2][kSelBins];
    __shared__ int s_scan[2][33];
    __shared__ __align__(16) uint32_t s_mine[kSelList], s_list[kSelList];
    __shared__ int s_digit, s_need, s_count, s_flag, s_top, s_cands, s_totals[3];
    __shared__ uint32_t s_prefix;
    grid_dependency_wait();
    grid_dependents_launch();
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = p.cluster, rank = blockIdx.x % C, pair = blockIdx.x / C;
    auto sync_all = [&] {
        if (C > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    auto remote = [&](auto *x, int k) { return C > 1 ? cluster.map_shared_rank(x, k) : x; };   // x of the CTA of rank k
    int32_t *s_pos = reinterpret_cast<int32_t *>(s_key + p.key_cap);
    const int b = pair / p.Hkv, g = pair % p.Hkv;
    const int tid = threadIdx.x, T = blockDim.x, warp = tid >> 5, lane = tid & 31;
    // this CTA's rows: row0 + i for i < cnt
    const int part = (p.rows.max_len + C - 1) / C, row0 = min(p.rows.max_len, rank * part);
    const int room = min(p.rows.max_len, row0 + part) - row0;
    const float *w = p.weights + static_cast<size_t>(pair) * p.wstride;
    const int32_t *pos = p.row_pos ? p.row_pos + static_cast<size_t>(pair) * p.wstride : nullptr;
    constexpr int kAhead = 8;
    float ahead_w[kAhead];   // the first rows' weights and positions come with the length: up to max_len they can be read
    int ahead_pos[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        const int i = tid + u * T;
        ahead_w[u] = i < room ? w[row0 + i] : 0.f;
        ahead_pos[u] = i < room && p.recent > 0 ? pos[row0 + i] : INT_MIN;
    }
    int n;
    bool ok = seq_rows_ok(p.rows, b, 0, n);
    if (tid == 0) {
        s_flag = 0;
        s_top = INT_MIN;
        s_cands = 0;
    }
    for (int i = tid; i < kSelBins; i += T) s_hist[0][i] = 0;
    __syncthreads();
    if (ok && n > p.budget && p.rows.pages != nullptr) {
        const int np = (n + p.rows.page_size - 1) / p.rows.page_size;
        for (int i = tid; i < np; i += T) {
            const int id = p.rows.pages[static_cast<size_t>(b) * p.rows.max_pages + i];
            if (id < 0 || id >= p.rows.num_pages) s_flag = 1;
        }
    }

    const int cnt = min(room, max(0, n - row0));
    float *nw = p.new_weights + static_cast<size_t>(pair) * p.new_wstride;
    int32_t *npos = p.new_row_pos ? p.new_row_pos + static_cast<size_t>(pair) * p.new_wstride : nullptr;
    const int left = min(n, p.budget);
    const bool selects = ok && n > p.budget;
    const int held = min(cnt, p.key_cap), held_pos = p.recent > 0 ? min(cnt, p.pos_cap) : 0;
    if (selects) {
        int top = INT_MIN;
        for (int i0 = tid; i0 < cnt; i0 += kAhead * T) {
            if (i0 != tid) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = i0 + u * T;
                    ahead_w[u] = i < held ? w[row0 + i] : 0.f;
                    ahead_pos[u] = i < cnt && p.recent > 0 ? pos[row0 + i] : INT_MIN;
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * T;
                if (i < held) s_key[i] = evict_key(ahead_w[u], false);
                if (i < held_pos) s_pos[i] = ahead_pos[u];
                if (i < cnt) top = max(top, ahead_pos[u]);
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0 && p.recent > 0) atomicMax(&s_top, top);
    }
    sync_all();
    ok = ok && s_flag == 0;
    if (tid == 0 && rank == 0) {
        if (g == 0) {
            p.new_seqlens[b] = ok ? min(n, p.budget) : n;
            if (!ok) atomicOr(p.err, kErrInput);
        }
        if (!p.fused) p.counts[pair] = 0;
    }
    long long newest = s_top;
    if (C > 1 && selects && p.recent > 0)
        for (int k = 0; k < C; ++k) newest = max(newest, static_cast<long long>(*remote(&s_top, k)));
    if (ok && p.copy)
        for (int r = rank * T + tid; r < left; r += C * T) {
            nw[r] = w[r];
            if (npos) npos[r] = pos[r];
        }
    if (!ok || n <= p.budget) {   // nothing of a sequence that breaks its bounds is touched
        if (C > 1) cluster.sync();   // others may still look at s_top
        return;
    }

    auto is_recent = [&](int at) { return static_cast<long long>(at) > newest - p.recent; };
    auto key = [&](int i) {
        return i < held ? s_key[i] : evict_key(w[row0 + i], p.recent > 0 && is_recent(pos[row0 + i]));
    };

    // ---- prefix = the budget-th greatest key, need = its rank among its equals
    uint32_t prefix = 0;
    int need = p.budget;
    // The bin of the need-th greatest key of histogram h, summed over the first `ctas` CTAs' (each finds the same), or of
    // this CTA's alone (ctas = 1).
    auto find_bin = [&](int h, int ctas) {
        constexpr int kPer = 8;   // kSelBins / 256 threads
        const int per = kSelBins / T, low = kSelBins - (tid + 1) * per;   // this thread's bins low .. low + per - 1
        int count[kPer] = {}, sum = 0;
#pragma unroll 1
        for (int k0 = 0; k0 < ctas; k0 += 4) {
            int2 x[4][kPer / 2];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i)
                    x[k][i] = k0 + k < ctas && 2 * i < per
                                  ? *reinterpret_cast<const int2 *>((ctas > 1 ? remote(&s_hist[h][0], k0 + k) : &s_hist[h][0]) + low + 2 * i)
                                  : make_int2(0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) {
                    count[2 * i] += x[k][i].x;
                    count[2 * i + 1] += x[k][i].y;
                }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum += count[i];
        int total;
        int before = block_scan(sum, s_scan[0], total);
        if (before < need && need <= before + sum) {
            bool found = false;
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i) {   // from the greatest
                if (i >= per || found) continue;
                if (need <= before + count[i]) {
                    s_digit = low + i;
                    s_need = need - before;
                    s_count = count[i];
                    found = true;
                }
                before += count[i];
            }
        }
        __syncthreads();
        need = s_need;
    };
    int recents = 0;   // the recent rows' keys become the greatest, and are counted apart: all in one bin
    for (int i0 = tid; i0 < cnt; i0 += kAhead * T) {
        uint32_t x[kAhead];
        int at[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * T;
            x[u] = i < cnt ? (i < held ? s_key[i] : evict_key(w[row0 + i], false)) : 0u;
            at[u] = i < cnt && p.recent > 0 ? (i < held_pos ? s_pos[i] : pos[row0 + i]) : INT_MIN;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * T;
            if (i >= cnt) continue;
            if (p.recent > 0 && is_recent(at[u])) {
                if (i < held) s_key[i] = 0xffffffffu;
                ++recents;
            } else {
                atomicAdd(&s_hist[0][x[u] >> 21], 1);
            }
        }
    }
    recents = __reduce_add_sync(0xffffffffu, recents);
    if (lane == 0 && recents) atomicAdd(&s_hist[0][kSelBins - 1], recents);
    sync_all();
    find_bin(0, C);
    prefix = static_cast<uint32_t>(s_digit) << 21;
    const int count = s_count;
    if (count <= kSelList) {   // the bin's keys, from all CTAs
#pragma unroll 4
        for (int i = tid; i < cnt; i += T) {
            const uint32_t x = key(i);
            if (x >> 21 == prefix >> 21) s_mine[atomicAdd(&s_cands, 1)] = x;
        }
        sync_all();
        for (int k = 0, at = 0; k < C; ++k) {
            const int m = *remote(&s_cands, k);
            const uint32_t *from = remote(&s_mine[0], k);
            for (int i = tid; i < m; i += T) s_list[at + i] = from[i];
            at += m;
        }
        if (count <= kSelRank) {
            __syncthreads();
            if (tid < count) {
                const uint32_t x = s_list[tid];
                int above = 0, same = 0;
#pragma unroll 4
                for (int i = 0; i < count; ++i) {
                    above += s_list[i] > x;
                    same += s_list[i] == x;
                }
                if (above < need && need <= above + same) {   // every equal key writes the same
                    s_prefix = x;
                    s_need = need - above;
                }
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
        } else {
#pragma unroll 1
            for (int pass = 1; pass < 3; ++pass) {
                const int prev = pass == 1 ? 21 : 10, shift = pass == 1 ? 10 : 0;
                for (int i = tid; i < kSelBins; i += T) s_hist[1][i] = 0;
                __syncthreads();
                for (int i = tid; i < count; i += T) {
                    const uint32_t x = s_list[i];
                    if (x >> prev == prefix >> prev) atomicAdd(&s_hist[1][(x >> shift) & ((1u << (prev - shift)) - 1)], 1);
                }
                __syncthreads();
                find_bin(1, 1);
                prefix |= static_cast<uint32_t>(s_digit) << shift;
            }
        }
    } else {
#pragma unroll 1
        for (int pass = 1; pass < 3; ++pass) {
            const int h = pass & 1, prev = pass == 1 ? 21 : 10, shift = pass == 1 ? 10 : 0;
            for (int i = tid; i < kSelBins; i += T) s_hist[h][i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int i = tid; i < cnt; i += T) {
                const uint32_t x = key(i);
                if (x >> prev == prefix >> prev) atomicAdd(&s_hist[h][(x >> shift) & ((1u << (prev - shift)) - 1)], 1);
            }
            sync_all();
            find_bin(h, C);
            prefix |= static_cast<uint32_t>(s_digit) << shift;
        }
    }
    // rows above `prefix` stay, and the first `need` of those equal to it

    // ---- holes and movers, each thread over rows [lo, hi) of its CTA's
    const int per = (cnt + T - 1) / T | 1;
    const int lo = min(cnt, tid * per), hi = min(cnt, lo + per);
    int eq = 0, holes = 0, movers = 0, total;
#pragma unroll 4
    for (int i = lo; i < hi; ++i) eq += key(i) == prefix;
    int eq0 = block_scan(eq, s_scan[0], total);
    auto before_ranks = [&](int which) {   // what the CTAs of lower rank counted
        int sum = 0;
        for (int k = 0; k < rank; ++k) sum += *remote(&s_totals[which], k);
        return sum;
    };
    if (C > 1) {
        if (tid == 0) s_totals[0] = total;
        cluster.sync();
        eq0 += before_ranks(0);
    }
    int run = eq0;
#pragma unroll 4
    for (int i = lo; i < hi; ++i) {
        const uint32_t x = key(i);
        const bool same = x == prefix, keep = x > prefix || (same && run < need);
        run += same;
        holes += !keep && row0 + i < p.budget;
        movers += keep && row0 + i >= p.budget;
    }
    int moved;
    int at_hole = block_scan(holes, s_scan[0], total);
    int at_mover = block_scan(movers, s_scan[1], moved);
    if (C > 1) {
        if (tid == 0) {
            s_totals[1] = total;
            s_totals[2] = moved;
        }
        cluster.sync();
        at_hole += before_ranks(1);
        at_mover += before_ranks(2);
        moved = 0;
        for (int k = 0; k < C; ++k) moved += *remote(&s_totals[2], k);
    }
    int32_t *src = p.moves + static_cast<size_t>(pair) * 2 * p.move_cap, *dst = src + p.move_cap;
    if (holes + movers > 0) {
        run = eq0;
        for (int i = lo; i < hi; ++i) {
            const uint32_t x = key(i);
            const bool same = x == prefix, keep = x > prefix || (same && run < need);
            run += same;
            if (!keep && row0 + i < p.budget) dst[at_hole++] = row0 + i;
            if (keep && row0 + i >= p.budget) src[at_mover++] = row0 + i;
        }
    }
    sync_all();   // the lists (and the copied metadata) are written, and nobody reads another's shared memory any more
    for (int i = rank * T + tid; i < moved; i += C * T) {
        nw[dst[i]] = w[src[i]];
        if (npos) npos[dst[i]] = pos[src[i]];
    }
    if (p.fused)
        evict_move<KIND>(p, b, g, src, dst, moved, rank * (T / 32) + warp, C * (T / 32), lane);
    else if (tid == 0 && rank == 0)
        p.counts[pair] = moved;
}

// The listed rows of all (sequence, KV head) pairs, 8 warps a CTA.  Bound by memory: a row is read and written once
// (bf16: 110 MB in 16 us; in 4 bits a row is 13 sectors of 32 B for 136 B, 31 MB in 18 us).
template <int KIND>
__global__ void __launch_bounds__(256) kv_move_kernel(const __grid_constant__ KvEvictParams p) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv;
    const int32_t *src = p.moves + static_cast<size_t>(blockIdx.x) * 2 * p.move_cap;
    evict_move<KIND>(p, b, g, src, src + p.move_cap, p.counts[blockIdx.x], blockIdx.y * 8 + (threadIdx.x >> 5),
                     gridDim.y * 8, threadIdx.x & 31);
}

}  // namespace gqa
