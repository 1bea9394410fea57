// i8ffn_few.hpp -- the INT8 feed-forward operators for up to 16 tokens: kernels
// that stream the live experts' weights (or the dense front's) once.
//
// Bound: the weights' bytes from HBM.  An item is a wave's own: 4 x RG weight
// rows over the whole of K, so no wave waits for another and a wave's next item
// is requested while its last one is multiplied.  The front's 4 rows are gate
// and up of two outputs, the down projection's 4 adjacent outputs.
//
// v_mfma_i32_4x4x4_16b_i8 multiplies 16 blocks of 4 rows x 4 columns, 4 K each.
// A lane holds 4 K of row (or column) lane % 4 for block lane / 4, so with block
// b at the 16-byte chunk b of 256 bytes a load instruction of the weights takes
// 4 rows x 256 contiguous bytes (whole lines), one of the codes 4 tokens x 256
// bytes, and both feed the matrix core as they come, 4 products of 4 bytes
// each: no transpose through LDS, and the 16 partial sums of an output are added
// once an item.  A column without a token multiplies another token's codes; it
// is never stored.
//
// Codes are in LDS: either each workgroup quantises the rows for itself while its
// first weights travel (few rows: that costs less than a launch), or they were
// written by a kernel ahead and are copied.
#pragma once
#include <type_traits>

#include "i8ffn_device.hpp"

namespace qlin {

constexpr int kFewPairs = 256;   // 16 tokens, 16 slots
constexpr int kFewThreads = 512, kFewWaves = kFewThreads / 64;
constexpr int kFewTokens = 16;   // tokens of a chunk: four columns sets

typedef int i32x4f_t __attribute__((ext_vector_type(4)));

// Pairs by expert, in chunks of up to `cap` pairs of one expert (at most kFewTokens).
struct FewList {
    int chunks;
    int expert[kFewPairs], first[kFewPairs], count[kFewPairs];  // of each chunk
    int pair[kFewPairs];                                        // pairs in expert order, pair order inside
};

// Built by a whole workgroup from the pairs' experts (ids outside [0, E) are in no chunk).  Every thread owns a
// pair and counts those ahead of it: pairs of lower experts, and earlier ones of its own.  Opens and ends with a
// barrier; sid keeps each pair's expert, -1 where it has none.
__device__ __forceinline__ void few_list(FewList& l, int* sid, int npairs, const int32_t* ids, int E, int cap) {
    const int tid = threadIdx.x;
    int e = -1;
    if (tid < npairs) {
        e = ids[tid];
        e = (uint32_t)e < (uint32_t)E ? e : -1;
    }
    if (tid < kFewPairs) sid[tid] = e;
    if (tid == 0) l.chunks = 0;
    w4_lds_barrier();
    int lower = 0, before = 0, all = 0, heads = 0;
    if (tid < npairs) {
        typedef int i32x4l_t __attribute__((ext_vector_type(4)));
#pragma unroll 4
        for (int q = 0; q < npairs; q += 4) {
            const i32x4l_t o = *(const i32x4l_t*)(sid + q);  // -1 past npairs
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lower += (uint32_t)o[i] < (uint32_t)e ? 1 : 0;  // as unsigned, -1 is never lower
                before += (o[i] == e && q + i < tid) ? 1 : 0;
                all += o[i] == e ? 1 : 0;
            }
        }
        if (e >= 0) {
            l.pair[lower + before] = tid;
            if (before == 0) l.first[lower] = all;  // for now: at the place of its first pair an expert's count
        }
    }
    w4_lds_barrier();
    const bool head = e >= 0 && before == 0;
    if (head) {
        for (int at = 0; at < lower;) {  // chunks of the experts ahead
            const int n = l.first[at];
            heads += (n + cap - 1) / cap;
            at += n;
        }
    }
    w4_lds_barrier();
    if (head) {
        const int n = (all + cap - 1) / cap;
        for (int c = 0; c < n; ++c) {
            l.expert[heads + c] = e;
            l.first[heads + c] = lower + c * cap;
            l.count[heads + c] = all - c * cap < cap ? all - c * cap : cap;
        }
        atomicMax(&l.chunks, heads + n);
    }
    w4_lds_barrier();
}

// sum over the 16 blocks: lanes of equal lane % 4; every lane gets it
__device__ __forceinline__ int blocks_sum(int v) {
    v += dpp_mov<0x128>(v);
    v += dpp_mov<0x124>(v);
    uint32_t a = (uint32_t)v, b = (uint32_t)v;
    swap32(a, b);
    a = b = a + b;
    swap16(a, b);
    return (int)(a + b);
}

// Steps of 256 K that a wave's loads are ahead of its products.
constexpr int kFewDepth = 4;

// LDS pitch of a code row: whole turns of the loads' ring, and the four tokens of a column set 64 bytes (16 banks) apart
__host__ __device__ constexpr int few_pitch(int K) { return (K + 256 * kFewDepth - 1) / (256 * kFewDepth) * (256 * kFewDepth) + 64; }

// Where the codes come from.
enum FewSrc { kFewQuantise = 0, kFewStaged = 1 };

// A workgroup quantises up to kFewUnits x 512 elements into its LDS: a unit is 512 elements of one row, one load a
// lane.  The loads are issued by the constructor, long before their use.
constexpr int kFewUnitsPerWave = 8, kFewUnits = kFewUnitsPerWave * kFewWaves;

template <int T>
struct FewQuantiser {
    u32x4_t v[kFewUnitsPerWave];
    int rows, K, segs, lane, wv;

    __device__ FewQuantiser(const uint16_t* x, int64_t ldx, int rows_, int K_)
        : rows(rows_), K(K_), segs((K_ + 511) >> 9), lane(threadIdx.x & 63),
          wv(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {
#pragma unroll
        for (int i = 0; i < kFewUnitsPerWave; ++i) {
            const int u = wv + i * kFewWaves, m = u / segs, k = (u - m * segs) * 512 + lane * 8;
            v[i] = u < rows * segs && k < K ? ld16(x + m * ldx + k) : u32x4_t{0, 0, 0, 0};
        }
    }
    // mag: one zeroed word a row
    __device__ void maxima(uint32_t* mag) const {
#pragma unroll
        for (int i = 0; i < kFewUnitsPerWave; ++i) {
            const int u = wv + i * kFewWaves;
            if (u >= rows * segs) break;  // uniform
            const uint32_t m = wave_mag(mag8(v[i], 0));
            if (lane == 0) atomicMax(&mag[u / segs], m);
        }
    }
    // after a barrier; zeros from K to the pitch
    __device__ void codes(const uint32_t* mag, int8_t* out, float* scale, int pitch) const {
#pragma unroll
        for (int i = 0; i < kFewUnitsPerWave; ++i) {
            const int u = wv + i * kFewWaves;
            if (u >= rows * segs) break;  // uniform
            const int m = u / segs, seg = u - m * segs, k = seg * 512 + lane * 8;
            double r;
            const float s = row_scale<T>(mag[m], r);
            if (seg == 0 && lane == 0) scale[m] = s;
            if (k < pitch) *(uint2*)(out + m * pitch + k) = codes8<T>(v[i], r);  // past K: zeros give zeros
        }
        const int done = segs * 512;  // the rest of the ring's turn
        for (int m = wv; m < rows; m += kFewWaves)
            for (int k = done + lane * 8; k < pitch; k += 512) *(uint2*)(out + m * pitch + k) = make_uint2(0u, 0u);
    }
};

// Copies code rows (row r is xq's row of[r], or r) to LDS.
__device__ __forceinline__ void stage_codes(const int8_t* xq, int64_t ldxq, const int* of, int rows, int K, int pitch,
                                            int8_t* out) {
    const int per = pitch / 16, total = rows * per;
    for (int i0 = threadIdx.x; i0 < total; i0 += 8 * kFewThreads) {
        u32x4_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kFewThreads, m = i / per, k = (i - m * per) * 16;
            v[j] = i < total && k < K ? ld16(xq + (of ? of[m] : m) * ldxq + k) : u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kFewThreads, m = i / per, k = (i - m * per) * 16;
            if (i < total) *(u32x4_t*)(out + m * pitch + k) = v[j];
        }
    }
}

// What a wave has requested: the first kFewDepth steps of its item, and the item's channel scales.  The ring is
// always full: the steps past an item's end are the next item's first.
struct FewRing {
    u32x4_t w[kFewDepth];
    f32x2v_t sc;
    const int8_t* wp;

    __device__ void prime(const int8_t* row, int K) {
        const int at = ((threadIdx.x & 63) >> 2) * 16;
        wp = row;
#pragma unroll
        for (int u = 0; u < kFewDepth; ++u) {
            const int k = u * 256 + at;
            w[u] = ld_stream(wp + (k < K ? k : 0));  // past K: any of the row, against zero codes
        }
    }
};

// One item: its sums with NS x 4 columns, cb[n] the code row (LDS, zeros past K) of this lane's token of set n.
template <int NS>
__device__ __forceinline__ void few_item(FewRing& ring, const int8_t* next, int K, const int8_t* const (&cb)[4],
                                         i32x4f_t (&acc)[4]) {
    constexpr int D = kFewDepth;
    const int at = ((threadIdx.x & 63) >> 2) * 16;
    const int turns = (K + 256 * D - 1) / (256 * D);
#pragma unroll
    for (int n = 0; n < NS; ++n) acc[n] = i32x4f_t{0, 0, 0, 0};
    for (int t = 0; t < turns; ++t) {
        int k0 = (t + 1) * 256 * D;  // of the ring's next turn
        if (t + 1 == turns) {
            k0 = 0;
            ring.wp = next;
        }
#pragma unroll
        for (int u = 0; u < D; ++u) {
            u32x4_t x[NS];
#pragma unroll
            for (int n = 0; n < NS; ++n) x[n] = *(const u32x4_t*)(cb[n] + (t * D + u) * 256 + at);
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    acc[n] = __builtin_amdgcn_mfma_i32_4x4x4i8((int)ring.w[u][d], (int)x[n][d], acc[n], 0, 0, 0);
            const int k = k0 + u * 256 + at;
            ring.w[u] = ld_stream(ring.wp + (k < K ? k : 0));
        }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[n][r] = blocks_sum(acc[n][r]);
}

// A wave's items [item, stop) of a list of chunks x `per` items.  enter(c): the chunk's weights; row(i), scales(i): the
// row that this lane loads of item i of the chunk entered last, and its channel scales; tokens(c, cb): looks up
// chunk c's tokens and returns their number; done(i, acc, sc).  The next item's rows are requested, and its scales,
// while this one is multiplied, across chunks too.
struct FewWork {
    int item, stop, per, c, i;

    template <class Enter, class Row, class Scales>
    __device__ void prime(FewRing& ring, int K, const Enter& enter, const Row& row, const Scales& scales) {
        if (item >= stop) return;
        c = item / per;
        i = item - c * per;
        enter(c);
        ring.sc = scales(i);
        ring.prime(row(i), K);
    }
    template <class Enter, class Row, class Scales, class Tokens, class Done>
    __device__ void run(FewRing& ring, int K, const Enter& enter, const Row& row, const Scales& scales,
                        const Tokens& tokens, const Done& done) {
        const int8_t* cb[4];
        int at = -1, cnt = 0;
        for (; item < stop; ++item) {
            if (c != at) cnt = tokens(c, cb);
            at = c;
            const int here = i;
            if (item + 1 < stop && ++i == per) {  // past the end: this item's rows, again
                i = 0;
                enter(++c);
            }
            const int8_t* next = row(i);
            const f32x2v_t sc = scales(i);
            i32x4f_t acc[4];
            if (cnt <= 4) few_item<1>(ring, next, K, cb, acc);
            else if (cnt <= 8) few_item<2>(ring, next, K, cb, acc);
            else few_item<4>(ring, next, K, cb, acc);
            done(here, acc, ring.sc);
            ring.sc = sc;
        }
    }
};

struct FewFrontParams {
    const uint16_t* x; int64_t ldx;                  // quantise: 16-bit rows
    const int8_t* xq; int64_t ldxq; const float* xs; // else: codes, scales
    int8_t* xq_out; float* xs_out;                   // dense, quantise: the codes and scales go here too
    int M, K;
    const float* logits; int64_t ldl; int E, topk, route;  // E = 0: dense
    int32_t* ids; float* gw;                         // with logits written, else read
    const int8_t* w; int64_t ldw; int64_t I; const float* ws; int ws_step; int act;
    uint16_t* y; int64_t ldy;                        // rows: pairs, or tokens where dense
};

// Workgroup b of G owns the items [b n / G, (b + 1) n / G) of all chunks' output
// pairs, each wave a run of them.
template <int T, int SRC, int NR>
__global__ __launch_bounds__(kFewThreads, 4) void few_front_kernel(const FewFrontParams p) {
    extern __shared__ __align__(16) uint8_t few_lds[];  // codes [M][pitch]
    __shared__ FewList list;
    __shared__ __align__(16) int sid[kFewPairs];
    __shared__ float scale[kFewTokens];
    __shared__ uint32_t mag[kFewTokens];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pitch = few_pitch(p.K);
    const bool moe = p.E > 0;
    int8_t* codes = (int8_t*)few_lds;
    const int npairs = moe ? p.M * p.topk : p.M;
    FewQuantiser<T> quant(p.x, p.ldx, SRC == kFewQuantise ? p.M : 0, p.K);
    if (tid < kFewTokens) mag[tid] = 0;
    if (moe && p.logits) {
        for (int m = wv; m < p.M; m += kFewWaves) {
            int id;
            float w;
            route_token<NR>(p.logits + m * p.ldl, p.E, p.topk, p.route, lane, id, w);
            if (lane < p.topk) {
                list.pair[m * p.topk + lane] = id;  // not yet in use
                if (blockIdx.x == 0) {
                    p.ids[m * p.topk + lane] = id;
                    p.gw[m * p.topk + lane] = w;
                }
            }
        }
    }
    __syncthreads();
    int chunks = 1;
    if (moe) {
        few_list(list, sid, npairs, p.logits ? (const int32_t*)list.pair : p.ids, p.E, kFewTokens);
        chunks = __builtin_amdgcn_readfirstlane(list.chunks);
    }
    FewWork work;
    work.per = (int)((p.I + 1) / 2);  // items of a chunk: two outputs
    const int n = chunks * work.per, waves = gridDim.x * kFewWaves, me = blockIdx.x * kFewWaves + wv;
    work.item = (int)((int64_t)n * me / waves);
    work.stop = (int)((int64_t)n * (me + 1) / waves);
    const int r4 = lane & 3, o = (lane >> 2) & 1;
    const int8_t* w = nullptr;
    const float* ws = nullptr;
    auto enter = [&](int c) {
        const int e = moe ? __builtin_amdgcn_readfirstlane(list.expert[c]) : 0;
        w = p.w + (int64_t)e * 2 * p.I * p.ldw;
        ws = p.ws + (int64_t)e * 2 * p.I * p.ws_step;
    };
    auto row = [&](int it) {  // gate rows of outputs 2 it and 2 it + 1, then their up rows
        const int64_t i = 2 * (int64_t)it + (r4 & 1), ic = i < p.I ? i : p.I - 1;
        return w + (ic + (r4 >> 1) * p.I) * p.ldw;
    };
    auto scales = [&](int it) {
        const int64_t i = 2 * (int64_t)it + o, ic = i < p.I ? i : p.I - 1;
        return f32x2v_t{ws[ic * p.ws_step], ws[(p.I + ic) * p.ws_step]};
    };
    FewRing ring;
    work.prime(ring, p.K, enter, row, scales);
    if constexpr (SRC == kFewQuantise) {
        quant.maxima(mag);
        w4_lds_barrier();
        quant.codes(mag, codes, scale, pitch);
        w4_lds_barrier();
        if (p.xq_out && blockIdx.x == 0) {
            for (int i = tid; i < p.M * (p.K / 16); i += kFewThreads) {
                const int m = i / (p.K / 16), k = (i - m * (p.K / 16)) * 16;
                *(u32x4_t*)(p.xq_out + m * p.ldxq + k) = *(const u32x4_t*)(codes + m * pitch + k);
            }
            if (tid < p.M) p.xs_out[tid] = scale[tid];
        }
    } else {
        if (tid < p.M) scale[tid] = p.xs[tid];
        stage_codes(p.xq, p.ldxq, nullptr, p.M, p.K, pitch, codes);
        w4_lds_barrier();
    }
    int row_of[4], cnt = 0;
    float xs[4];
    auto tokens = [&](int c, const int8_t* (&cb)[4]) {
        cnt = moe ? __builtin_amdgcn_readfirstlane(list.count[c]) : p.M;
        const int first = moe ? list.first[c] : 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int j = s * 4 + r4 < cnt ? s * 4 + r4 : 0;
            row_of[s] = moe ? list.pair[first + j] : j;
            const int t = moe ? row_of[s] / p.topk : j;
            cb[s] = codes + t * pitch;
            xs[s] = scale[t];
        }
        return cnt;
    };
    auto done = [&](int it, i32x4f_t (&acc)[4], const f32x2v_t& sc) {
        const int64_t i = 2 * (int64_t)it + o;
        if (lane >= 8 || i >= p.I) return;
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (s * 4 + r4 < cnt)
                p.y[row_of[s] * p.ldy + i] = f32_to_h<T>(gated(o ? acc[s][1] : acc[s][0], o ? acc[s][3] : acc[s][2], xs[s],
                                                               sc[0], sc[1], p.act));
    };
    work.run(ring, p.K, enter, row, scales, tokens, done);
}

struct FewDownParams {
    const uint16_t* h;                              // quantise: [P][I]
    const int8_t* hq; const float* hs;              // else: codes [P][I], scales
    int M, I;
    const int32_t* ids; const float* gw; int E, topk;
    const int8_t* w; int64_t ldw; int64_t H; const float* ws;
    uint16_t* y; int64_t ldy;
    int block;                                      // row groups whose sums LDS holds at once
    int rows;                                       // code rows that LDS holds at once
};

// Workgroup b of G owns a run of the output's 4-row groups and takes all
// experts through it, so the slots are joined in LDS, in slot order.  Where LDS
// does not hold all pairs' codes, the chunks are taken in batches that it holds.
template <int T, int SRC>
__global__ __launch_bounds__(kFewThreads, 4) void few_down_kernel(const FewDownParams p) {
    extern __shared__ __align__(16) uint8_t few_lds[];  // sums [block][P][4], then codes [rows][pitch]
    __shared__ FewList list;
    __shared__ __align__(16) int sid[kFewPairs];
    __shared__ float scale[kFewPairs];
    __shared__ uint32_t mag[kFewPairs];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int npairs = p.M * p.topk, pitch = few_pitch(p.I);
    float* sums = (float*)few_lds;
    int8_t* codes = (int8_t*)few_lds + (size_t)p.block * npairs * 16;
    FewQuantiser<T> quant(p.h, p.I, SRC == kFewQuantise ? npairs : 0, p.I);
    if (tid < kFewPairs) mag[tid] = 0;
    few_list(list, sid, npairs, p.ids, p.E, p.rows < kFewTokens ? p.rows : kFewTokens);
    const int chunks = __builtin_amdgcn_readfirstlane(list.chunks);
    const int groups = (int)(p.H / 4);
    const int g0 = (int)((int64_t)groups * blockIdx.x / gridDim.x), g1 = (int)((int64_t)groups * (blockIdx.x + 1) / gridDim.x);
    const int r4 = lane & 3;
    // the block of row groups, and the batch of chunks [c0, c1) with pairs from list.pair[base], that are worked on
    int gb = g0, nb = 0, c0 = 0, c1 = 0, base = 0, pairs = 0;
    const int8_t* w = nullptr;
    const float* ws = nullptr;
    auto row = [&](int it) { return w + (int64_t)4 * it * p.ldw; };
    auto scales = [&](int it) { return f32x2v_t{ws[4 * it], 0.f}; };
    auto enter = [&](int c) {
        const int e = __builtin_amdgcn_readfirstlane(list.expert[c0 + c]);
        w = p.w + ((int64_t)e * p.H + 4 * gb + r4) * p.ldw;
        ws = p.ws + (int64_t)e * p.H + 4 * gb + ((lane >> 2) & 3);
    };
    FewRing ring;
    FewWork work;
    auto open_batch = [&]() {  // from chunk c0; its weights are requested
        nb = g1 - gb < p.block ? g1 - gb : p.block;
        c1 = c0;
        base = c0 < chunks ? __builtin_amdgcn_readfirstlane(list.first[c0]) : 0;
        pairs = 0;
        while (c1 < chunks) {
            const int n = __builtin_amdgcn_readfirstlane(list.count[c1]);
            if (pairs + n > p.rows) break;
            pairs += n;
            ++c1;
        }
        work.per = nb;
        const int n = (c1 - c0) * nb;
        work.item = n * wv / kFewWaves;
        work.stop = n * (wv + 1) / kFewWaves;
        work.prime(ring, p.I, enter, row, scales);
    };
    auto stage = [&]() { stage_codes(p.hq, p.I, list.pair + base, pairs, p.I, pitch, codes); };
    open_batch();
    if constexpr (SRC == kFewQuantise) {
        quant.maxima(mag);
        w4_lds_barrier();
        quant.codes(mag, codes, scale, pitch);
    } else {
        if (tid < npairs && sid[tid] >= 0) scale[tid] = p.hs[tid];
        stage();
    }
    w4_lds_barrier();
    int pair[4], cnt = 0;
    float hs[4];
    auto tokens = [&](int c, const int8_t* (&cb)[4]) {
        cnt = __builtin_amdgcn_readfirstlane(list.count[c0 + c]);
        const int first = list.first[c0 + c];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int j = first + (s * 4 + r4 < cnt ? s * 4 + r4 : 0);
            pair[s] = list.pair[j];
            hs[s] = scale[pair[s]];
            cb[s] = codes + (SRC == kFewQuantise ? pair[s] : j - base) * pitch;
        }
        return cnt;
    };
    auto done = [&](int it, i32x4f_t (&acc)[4], const f32x2v_t& sc) {
        const int r = lane >> 2;
        if (r >= 4) return;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int a = r == 0 ? acc[s][0] : (r == 1 ? acc[s][1] : (r == 2 ? acc[s][2] : acc[s][3]));
            if (s * 4 + r4 < cnt) sums[(it * npairs + pair[s]) * 4 + r] = ((float)a * hs[s]) * sc[0];
        }
    };
    for (;;) {
        work.run(ring, p.I, enter, row, scales, tokens, done);
        w4_lds_barrier();  // everyone is done with the codes, and the batch's sums are there
        const int gs = gb, ns = nb;
        const bool more = c1 < chunks, restage = more || c0 > 0;  // chunks of this block
        c0 = more ? c1 : 0;
        gb = more ? gb : gb + nb;
        const bool last = gb >= g1;
        if (!last) {
            open_batch();  // its first weights travel while the sums are joined
            if (SRC == kFewStaged && restage) stage();
        }
        if (!more)
            for (int i = tid; i < p.M * ns * 4; i += kFewThreads) {
                const int t = i / (ns * 4), r = i - t * ns * 4;  // r: row of the block
                float sum = 0.f;
                for (int j = 0; j < p.topk; ++j) {
                    const int q = t * p.topk + j;
                    if (sid[q] >= 0) sum = fmaf(p.gw[q], sums[((r >> 2) * npairs + q) * 4 + (r & 3)], sum);
                }
                p.y[t * p.ldy + 4 * gs + r] = f32_to_h<T>(sum);
            }
        if (last) break;
        w4_lds_barrier();
    }
}

}  // namespace qlin
