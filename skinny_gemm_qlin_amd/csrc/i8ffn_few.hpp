// i8ffn_few.hpp -- the INT8 feed-forward operators for up to 16 tokens: kernels
// that stream the live experts' weights (or the dense front's) once.
//
// Bound: the weights' bytes from HBM.  An item is 4 weight rows over the whole of
// K (front: gate and up of two outputs; down: 4 adjacent outputs).  A workgroup
// of 8 waves a compute unit has a run of the items of all live experts, dealt to
// its waves by turns of D x 256 K, so that every wave has as many as any other,
// to one; an item on the border of two waves is joined in LDS in whole numbers.
// A wave's loads run D steps ahead, across items, and are not drained between
// them: the last turn of an item requests the first of the next.  (They are where
// the down projection goes on to another block of row groups or batch of codes.)
// 16 waves a compute unit, two workgroups, or items that are a wave's own were
// slower (one token, 2 x 14336 x 4096: 25.5 us with whole items, 19.5 us now, 117
// MB at 6.0 TB/s, as a kernel that only loads them).  64 experts top 6, 7168 x
// 2048, front and down: one token 31.9 + 19.9 us (5.5 and 4.4 TB/s; loads alone
// 27.5 + 15.4), of which 6 and 5 go by before the first product (routing, list,
// codes); 8 tokens 151 + 78 us (6.8 and 6.6 TB/s; loads alone 148 + 75).
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
// written by a kernel ahead and are copied.  The front's copy is not overlapped: the
// tokens' scales and the list are loaded behind it, loads come back in order, and so
// the first weights are requested when the codes have arrived.
#pragma once
#include <type_traits>

#include "i8ffn_device.hpp"
#include "i8ffn_plan.hpp"

namespace qlin {

typedef int i32x4f_t __attribute__((ext_vector_type(4)));

// x / d for 0 <= x < 2^24, r = 1 / d to within an ulp or two: the quotient of the floats is at most one off.
__device__ __forceinline__ int few_div(int x, int d, float r) {
    int q = (int)((float)x * r);
    q -= q * d > x ? 1 : 0;
    return q + ((q + 1) * d <= x ? 1 : 0);
}

// Pairs by expert, in chunks of up to `cap` pairs of one expert (at most kFewTokens).
struct FewList {
    int chunks, pairs, pad[2];
    i32x4f_t chunk[kFewPairs];              // expert, first pair, number of pairs
    int pair[kFewPairs], token[kFewPairs];  // pairs in expert order, pair order inside; their tokens
};

struct FewListTemp {
    int sid[kFewPairs];  // each pair's expert, -1 where it has none
    int meta[kFewPairs];
    int heads[4];
};

// Built by a whole workgroup from t.sid (-1 from npairs up to a multiple of 8; ready behind a barrier).  A pair's
// place is the number of pairs ahead of it, of lower experts and earlier ones of its own; two or four lanes count
// them.  Ends with a barrier.
__device__ __forceinline__ void few_list(FewList& l, FewListTemp& t, int npairs, int topk, int cap) {
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    typedef int i32x4l_t __attribute__((ext_vector_type(4)));
    const int sh = npairs <= kFewThreads / 4 ? 2 : 1, pr = tid >> sh, part = tid & ((1 << sh) - 1);
    const int e = pr < npairs ? t.sid[pr] : -1;
    int lower = 0, before = 0, all = 0;
    if (pr < npairs) {
#pragma unroll 2
        for (int q = part * 4; q < npairs; q += 4 << sh) {
            const i32x4l_t o = *(const i32x4l_t*)(t.sid + q);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lower += (uint32_t)o[i] < (uint32_t)e ? 1 : 0;  // as unsigned, -1 is never lower
                before += (o[i] == e && q + i < pr) ? 1 : 0;
                all += o[i] == e ? 1 : 0;
            }
        }
    }
    // over the pair's lanes: quad_perm 1 0 3 2, then 2 3 0 1
    lower += dpp_mov<0xB1>(lower);
    before += dpp_mov<0xB1>(before);
    all += dpp_mov<0xB1>(all);
    if (sh == 2) {
        lower += dpp_mov<0x4E>(lower);
        before += dpp_mov<0x4E>(before);
        all += dpp_mov<0x4E>(all);
    }
    if (tid < kFewPairs) t.meta[tid] = -1;
    w4_lds_barrier();
    if (e >= 0 && part == 0) {
        const int at = lower + before;
        l.pair[at] = pr;
        l.token[at] = few_div(pr, topk, __builtin_amdgcn_rcpf((float)topk));
        t.meta[at] = before | all << 16;
    }
    w4_lds_barrier();
    const int m = tid < kFewPairs ? t.meta[tid] : -1, b4 = m & 0xFFFF, cnt = m >> 16;
    const bool head = m >= 0 && b4 - few_div(b4, cap, __builtin_amdgcn_rcpf((float)cap)) * cap == 0;
    const uint64_t hm = __ballot(head);
    if (tid < kFewPairs && lane == 0) t.heads[wv] = __popcll(hm);
    w4_lds_barrier();
    if (head) {
        int c = __popcll(hm & ((1ull << lane) - 1ull));
        for (int q = 0; q < wv; ++q) c += t.heads[q];
        l.chunk[c] = i32x4f_t{t.sid[l.pair[tid]], tid, cnt - b4 < cap ? cnt - b4 : cap, 0};
    }
    if (tid == 0) l.chunks = t.heads[0] + t.heads[1] + t.heads[2] + t.heads[3];
    if (m >= 0 && (tid + 1 == kFewPairs || t.meta[tid + 1] < 0)) l.pairs = tid + 1;
    if (tid == 0 && m < 0) l.pairs = 0;
    w4_lds_barrier();
}

__device__ __forceinline__ void few_sid(FewListTemp& t, int npairs, const int32_t* ids, int E) {
    if (threadIdx.x < kFewPairs) {
        const int e = (int)threadIdx.x < npairs ? ids[threadIdx.x] : -1;
        t.sid[threadIdx.x] = (uint32_t)e < (uint32_t)E ? e : -1;
    }
}

// One workgroup: routes the tokens and leaves the pairs' experts in sid (before a barrier of the caller's).
template <int NR>
__device__ __forceinline__ void few_route(const float* logits, int64_t ldl, int M, int E, int topk, int route, int32_t* ids,
                                          float* gw, bool store, FewListTemp& t) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, npairs = M * topk;
    if (npairs + threadIdx.x < kFewPairs && threadIdx.x < 8) t.sid[npairs + threadIdx.x] = -1;
    for (int m = wv; m < M; m += kFewWaves) {
        int id;
        float w;
        route_token<NR>(logits + m * ldl, E, topk, route, lane, id, w);
        if (lane < topk) {
            t.sid[m * topk + lane] = id;
            if (store) {
                ids[m * topk + lane] = id;
                gw[m * topk + lane] = w;
            }
        }
    }
}

// Adds a wave's four accumulators over the 16 blocks: lane l gets the sum of row few_row(l), column l % 4.  Lanes 32
// and 16 apart first, where a swap and an addition put two accumulators' halves side by side.
__device__ __forceinline__ int blocks_sum(const i32x4f_t& acc) {
    uint32_t a = (uint32_t)acc[0], b = (uint32_t)acc[1], c = (uint32_t)acc[2], d = (uint32_t)acc[3];
    swap32(a, b);
    swap32(c, d);
    a += b;  // row 0 in lanes ..31, row 1 above
    c += d;  // row 2, row 3
    swap16(a, c);
    int v = (int)(a + c);  // rows 0, 2, 1, 3 in lanes 0.., 16.., 32.., 48..
    v += dpp_mov<0x128>(v);
    return v + dpp_mov<0x124>(v);
}
__device__ __forceinline__ int few_row(int lane) { return ((lane >> 4) & 1) * 2 + (lane >> 5); }

// Where the codes come from.
enum FewSrc { kFewQuantise = 0, kFewStaged = 1 };

// A workgroup quantises up to kFewUnits x 512 elements into its LDS: a unit is 512 elements of one row, one load a
// lane.  The loads are issued by the constructor, long before their use.
template <int T>
struct FewQuantiser {
    u32x4_t v[kFewUnitsPerWave];
    int rows, K, segs, units, lane, wv;
    float rseg;

    __device__ FewQuantiser(const uint16_t* x, int64_t ldx, int rows_, int K_)
        : rows(rows_), K(K_), segs((K_ + 511) >> 9), units(rows_ * segs), lane(threadIdx.x & 63),
          wv(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), rseg(__builtin_amdgcn_rcpf((float)segs)) {
#pragma unroll
        for (int i = 0; i < kFewUnitsPerWave; ++i) {
            v[i] = u32x4_t{0, 0, 0, 0};
            if (i * kFewWaves + wv >= units) break;  // uniform
            int m, seg;
            where(i, m, seg);
            const int k = seg * 512 + lane * 8;
            if (k < K) v[i] = ld16(x + m * ldx + k);
        }
    }
    __device__ void where(int i, int& m, int& seg) const {
        const int u = i * kFewWaves + wv;
        m = __builtin_amdgcn_readfirstlane(few_div(u, segs, rseg));
        seg = u - m * segs;
    }
    // mag: one zeroed word a row
    __device__ void maxima(uint32_t* mag) const {
#pragma unroll
        for (int i = 0; i < kFewUnitsPerWave; ++i) {
            if (i * kFewWaves + wv >= units) break;  // uniform
            int m, seg;
            where(i, m, seg);
            const uint32_t a = wave_mag(mag8(v[i], 0));
            if (lane == 0) atomicMax(&mag[m], a);
        }
    }
    // after a barrier; zeros from K to the pitch
    __device__ void codes(const uint32_t* mag, int8_t* out, float* scale, int pitch) const {
        int last = -1;
        RowScale o{};
#pragma unroll
        for (int i = 0; i < kFewUnitsPerWave; ++i) {
            if (i * kFewWaves + wv >= units) break;  // uniform
            int m, seg;
            where(i, m, seg);
            const int k = seg * 512 + lane * 8;
            if (m != last) {  // uniform
                o = row_scale<T>((uint32_t)__builtin_amdgcn_readfirstlane((int)mag[m]));
                if (lane == 0) scale[m] = o.s;  // every wave of the row writes the same
                last = m;
            }
            if (k < pitch) *(uint2*)(out + m * pitch + k) = codes8<T>(v[i], o);  // past K: zeros give zeros
        }
        const int done = segs * 512;  // the rest of the ring's turn
        for (int m = wv; m < rows; m += kFewWaves)
            for (int k = done + lane * 8; k < pitch; k += 512) *(uint2*)(out + m * pitch + k) = make_uint2(0u, 0u);
    }
};

__device__ const u32x4_t kFewZero16 = {0u, 0u, 0u, 0u};

// Copies code rows (row r is xq's row of[r], or r) to LDS, 1 KB a load instruction, zeros from K to the end of the last
// turn; the caller waits.
__device__ __forceinline__ void stage_codes(const int8_t* xq, int64_t ldxq, const int* of, int rows, int K, int pitch,
                                            int8_t* out) {
    const int lane = threadIdx.x & 63, span = pitch - 64;
    for (int r = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); r < rows; r += kFewWaves) {
        const int8_t* src = xq + (of ? __builtin_amdgcn_readfirstlane(of[r]) : r) * ldxq + lane * 16;
        for (int k = 0; k < span; k += 1024)
            if (k + lane * 16 < span)  // lanes past it write nothing
                __builtin_amdgcn_global_load_lds(k + lane * 16 < K ? (const void*)(src + k) : (const void*)&kFewZero16,
                                                 (lds_void_t*)(out + r * pitch + k), 16, 0, 0);
    }
}

// Everything but this wave's last N loads (its ring's) is there; behind the barrier what the others loaded into LDS, too.
template <int N>
__device__ __forceinline__ void few_staged_barrier() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x70);  // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// What a wave has requested: D steps (a turn) of its item, and the item's channel scales.  The ring is always full:
// behind an item's last turn follows the next item's first.
template <int D>
struct FewRing {
    u32x4_t w[D];
    f32x2v_t sc;
    const int8_t* wp;

    __device__ void prime(const int8_t* row, int turn, int K) {
        const int at = ((threadIdx.x & 63) >> 2) * 16;
        wp = row;
#pragma unroll
        for (int u = 0; u < D; ++u) {
            const int k = (turn * D + u) * 256 + at;
            w[u] = ld_stream(wp + (k < K ? k : 0));  // past K: any of the row, against zero codes
        }
    }
};

// Turns [t, end) of an item, at least one: this lane's sums (blocks_sum) with NS x 4 columns, cb[n] where in few_lds the code
// row of its token of set n lies (zeros past K).
template <int NS, int D>
__device__ __forceinline__ void few_item(FewRing<D>& ring, const int8_t* next, int t, int end, int K,
                                         const int (&cb)[NS], int (&sum)[NS]) {
    extern __shared__ __align__(16) uint8_t few_lds[];
    i32x4f_t acc[NS];
    const int at = ((threadIdx.x & 63) >> 2) * 16;
#pragma unroll
    for (int n = 0; n < NS; ++n) acc[n] = i32x4f_t{0, 0, 0, 0};
    do {
        int k0 = (t + 1) * 256 * D;  // of the ring's next turn
        if (t + 1 == end) {
            k0 = 0;
            ring.wp = next;
        }
        u32x4_t x[2][NS];  // codes of this step and the next
#pragma unroll
        for (int n = 0; n < NS; ++n) x[0][n] = *(const u32x4_t*)(few_lds + cb[n] + t * D * 256 + at);
#pragma unroll
        for (int u = 0; u < D; ++u) {
            if (u + 1 < D) {
#pragma unroll
                for (int n = 0; n < NS; ++n) x[(u + 1) & 1][n] = *(const u32x4_t*)(few_lds + cb[n] + (t * D + u + 1) * 256 + at);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    acc[n] = __builtin_amdgcn_mfma_i32_4x4x4i8((int)ring.w[u][d], (int)x[u & 1][n][d], acc[n], 0, 0, 0);
            const int k = k0 + u * 256 + at;
            ring.w[u] = ld_stream(ring.wp + (k < K ? k : 0));
            __builtin_amdgcn_sched_barrier(0);  // or the turn's loads are all issued at its end, when nothing is in flight
        }
    } while (++t < end);
#pragma unroll
    for (int n = 0; n < NS; ++n) sum[n] = blocks_sum(acc[n]);
}

// first of share `me`, where every share has q and the first r one more
__device__ __forceinline__ int few_first(int q, int r, int me) { return me * q + (me < r ? me : r); }

// Sums of the items that more than one wave had turns of: [wave that had its first turn][token][row], zeroed ahead.
typedef int FewSlots[kFewWaves][kFewTokens][4];

// A workgroup's items, chunks x `per` of them, are dealt to its waves by turns of D x 256 K: every wave has as many as
// any other, to one.  An item that lies on the border of two waves is joined in LDS, in whole numbers.
//   enter(c): the chunk's weights, and its FewChunk; row(i), scales(i): the row that this lane loads of item i of the
//   chunk entered last, and the channel scales that it needs; tokens(chunk, cb): looks up the tokens of a chunk;
//   done(i, sum, sc).
template <int NS, int D>
struct FewWork {
    int per, turns, q, r;      // items a chunk, turns an item; turns a wave, and how many waves have one more
    int c, i, t, left;         // chunk, item in it, turn of it; turns that are left
    i32x4f_t chunk;            // the chunk entered last
    int open_c, open_i;        // an item whose first turn was this wave's and whose last was not (open_c < 0: none)

    // items [first, first + items) of all
    template <class Enter, class Row, class Scales>
    __device__ void prime(FewRing<D>& ring, int first, int items, int wave, int K, const Enter& enter, const Row& row,
                          const Scales& scales) {
        turns = (K + 256 * D - 1) / (256 * D);
        q = items * turns / kFewWaves;
        r = items * turns % kFewWaves;
        const int at = few_first(q, r, wave);
        left = q + (wave < r ? 1 : 0);
        int it = few_div(at, turns, __builtin_amdgcn_rcpf((float)turns));
        t = at - it * turns;
        it = left > 0 ? first + it : first;  // without turns: any item, so that the loads are the same on all paths
        c = __builtin_amdgcn_readfirstlane(few_div(it, per, __builtin_amdgcn_rcpf((float)per)));
        i = __builtin_amdgcn_readfirstlane(it - c * per);
        t = __builtin_amdgcn_readfirstlane(left > 0 ? t : 0);
        left = __builtin_amdgcn_readfirstlane(left);
        open_c = -1;
        open_i = 0;
        chunk = enter(c);
        ring.sc = scales(i);
        ring.prime(row(i), t, K);
    }
    template <class Enter, class Row, class Scales, class Tokens, class Done>
    __device__ void run(FewRing<D>& ring, int wave, int K, FewSlots& slots, const Enter& enter, const Row& row,
                        const Scales& scales, const Tokens& tokens, const Done& done) {
        int cb[NS];
        const int lane = threadIdx.x & 63;
        int at = -1;
        while (left > 0) {
            if (c != at) tokens(chunk, cb);
            at = c;
            const int here = i, t0 = t, end = turns - t < left ? turns : t + left;
            left -= end - t0;
            if (left > 0 && ++i == per) {
                i = 0;
                chunk = enter(++c);
            }
            t = 0;
            // past the end: a turn of the chunk's first rows, the same for every wave that ends in it, which the L2s hold
            const int8_t* next = row(left > 0 ? i : 0);
            const f32x2v_t sc = scales(i);
            int sum[NS];
            few_item<NS, D>(ring, next, t0, end, K, cb, sum);
            if (t0 == 0 && end == turns) {
                done(here, sum, ring.sc);
            } else {
                int home = wave;
                if (t0 > 0) {  // the wave that has the item's first turn
                    const int tau = few_first(q, r, wave) - t0, big = r * (q + 1);
                    home = tau < big ? few_div(tau, q + 1, __builtin_amdgcn_rcpf((float)(q + 1)))
                                     : r + few_div(tau - big, q, __builtin_amdgcn_rcpf((float)q));
                } else {
                    open_c = at;
                    open_i = here;
                }
                if ((lane & 15) < 4)
#pragma unroll
                    for (int s = 0; s < NS; ++s) atomicAdd(&slots[home][s * 4 + (lane & 3)][few_row(lane)], sum[s]);
            }
            ring.sc = sc;
        }
    }
    // behind a barrier: the item that the wave had the first turn of
    template <class Enter, class Scales, class Tokens, class Done>
    __device__ void close(int wave, FewSlots& slots, const Enter& enter, const Scales& scales, const Tokens& tokens,
                          const Done& done) {
        if (open_c < 0) return;
        int cb[NS];
        const int lane = threadIdx.x & 63;
        int sum[NS];
        tokens(enter(open_c), cb);
#pragma unroll
        for (int s = 0; s < NS; ++s) sum[s] = slots[wave][s * 4 + (lane & 3)][few_row(lane)];
        done(open_i, sum, scales(open_i));
    }
};

__device__ __forceinline__ void few_clear(FewSlots& slots) {
    static_assert(sizeof(FewSlots) == kFewThreads * 4, "a word a thread");
    ((int*)slots)[threadIdx.x] = 0;
}

// share `me` of `of` equal ones of n
__device__ __forceinline__ void few_share(int n, int me, int of, int& first, int& count) {
    const int q = few_div(n, of, __builtin_amdgcn_rcpf((float)of)), r = n - q * of;
    first = __builtin_amdgcn_readfirstlane(few_first(q, r, me));
    count = __builtin_amdgcn_readfirstlane(q + (me < r ? 1 : 0));
}

// Staged sources: a kernel ahead quantises the rows (tokens or pairs), a workgroup
// a row, and one more workgroup routes and makes the list.
struct FewPrepParams {
    const uint16_t* x; int64_t ldx; int rows, K; int8_t* xq; int64_t ldxq; float* xs;
    bool pairs;                                      // rows are pairs: those without an expert are left out
    const float* logits; int64_t ldl; int M, E, topk, route, cap;
    int32_t* ids; float* gw; FewList* list;          // the list: by workgroup `rows`, if there is one
};

struct FewFrontParams {
    const uint16_t* x; int64_t ldx;                  // quantise: 16-bit rows
    const int8_t* xq; int64_t ldxq; const float* xs; // staged: codes, scales
    const FewList* list;                             // staged: of the pairs
    int8_t* xq_out; float* xs_out;                   // dense, quantise: the codes and scales go here too
    int M, K;
    const float* logits; int64_t ldl; int E, topk, route;  // E = 0: dense
    int32_t* ids; float* gw;                         // with logits written, else read
    const int8_t* w; int64_t ldw; int64_t I; const float* ws; int ws_step; int act;
    uint16_t* y; int64_t ldy;                        // rows: pairs, or tokens where dense
};

__device__ __forceinline__ void few_copy_list(FewList& to, const FewList* from) {
    for (int i = threadIdx.x; i < (int)(sizeof(FewList) / 16); i += kFewThreads)
        ((u32x4_t*)&to)[i] = ((const u32x4_t*)from)[i];
}

template <int T, int NR>
__global__ __launch_bounds__(kFewThreads) void few_prep_kernel(const FewPrepParams p) {
    if ((int)blockIdx.x < p.rows) {
        if (p.pairs && (uint32_t)p.ids[blockIdx.x] >= (uint32_t)p.E) return;
        quantise_row_wg<T, kFewThreads>(p.x + blockIdx.x * p.ldx, p.K, p.xq + blockIdx.x * p.ldxq, p.xs + blockIdx.x);
        return;
    }
    __shared__ __align__(16) FewList list;
    __shared__ __align__(16) FewListTemp temp;
    const int npairs = p.M * p.topk;
    if (p.logits) few_route<NR>(p.logits, p.ldl, p.M, p.E, p.topk, p.route, p.ids, p.gw, true, temp);
    else few_sid(temp, npairs, p.ids, p.E);
    w4_lds_barrier();
    few_list(list, temp, npairs, p.topk, p.cap);
    for (int i = threadIdx.x; i < (int)(sizeof(FewList) / 16); i += kFewThreads)
        ((u32x4_t*)p.list)[i] = ((const u32x4_t*)&list)[i];
}

// A workgroup owns a run of all chunks' items, two outputs each.
// NR: only where the workgroup routes.
template <int T, int SRC, int NS, int D, int NR>
__global__ __launch_bounds__(kFewThreads, 2) void few_front_kernel(const FewFrontParams p) {
    extern __shared__ __align__(16) uint8_t few_lds[];  // codes [M][pitch]
    __shared__ __align__(16) FewList list;
    __shared__ __align__(16) FewListTemp temp;
    __shared__ __align__(16) FewSlots slots;
    __shared__ float scale[kFewTokens];
    __shared__ uint32_t mag[kFewTokens];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pitch = few_pitch(p.K, D);
    const bool moe = p.E > 0;
    int8_t* codes = (int8_t*)few_lds;
    const int npairs = moe ? p.M * p.topk : p.M;
    FewQuantiser<T> quant(p.x, p.ldx, SRC == kFewQuantise ? p.M : 0, p.K);
    few_clear(slots);
    if constexpr (SRC == kFewQuantise) {
        if (tid < kFewTokens) mag[tid] = 0;
        if (moe) {
            if (p.logits) few_route<NR>(p.logits, p.ldl, p.M, p.E, p.topk, p.route, p.ids, p.gw, blockIdx.x == 0, temp);
            else few_sid(temp, npairs, p.ids, p.E);
        }
        w4_lds_barrier();
        if (moe) few_list(list, temp, npairs, p.topk, 4 * NS);
    } else {
        stage_codes(p.xq, p.ldxq, nullptr, p.M, p.K, pitch, codes);
        if (tid < p.M) scale[tid] = p.xs[tid];
        if (moe) {
            few_copy_list(list, p.list);
            w4_lds_barrier();
        }
    }
    const int chunks = moe ? __builtin_amdgcn_readfirstlane(list.chunks) : 1;
    FewWork<NS, D> work;
    work.per = (int)((p.I + 1) / 2);  // items of a chunk
    int first_item, items;
    few_share(chunks * work.per, blockIdx.x, gridDim.x, first_item, items);
    const int r4 = lane & 3, o = lane >> 5, I = (int)p.I;
    const int8_t* w = nullptr;
    const float* ws = nullptr;
    auto enter = [&](int c) {
        const i32x4f_t h = moe && chunks > 0 ? list.chunk[c] : i32x4f_t{0, 0, p.M, 0};
        const int e = __builtin_amdgcn_readfirstlane(h[0]);
        w = p.w + (int64_t)e * 2 * p.I * p.ldw;
        ws = p.ws + (int64_t)e * 2 * p.I * p.ws_step;
        return h;
    };
    auto row = [&](int it) {  // gate rows of outputs 2 it and 2 it + 1, then their up rows
        const int i = 2 * it + (r4 & 1), ic = i < I ? i : I - 1;
        return w + (uint64_t)(uint32_t)(ic + (r4 >> 1) * I) * (uint32_t)p.ldw;
    };
    auto scales = [&](int it) {
        const int i = 2 * it + o, ic = i < I ? i : I - 1;
        return f32x2v_t{ws[ic * p.ws_step], ws[(I + ic) * p.ws_step]};
    };
    FewRing<D> ring;
    work.prime(ring, items > 0 ? first_item : 0, items, wv, p.K, enter, row, scales);
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
        few_staged_barrier<D>();
    }
    int row_of[NS], cnt = 0;
    float xs[NS];
    auto tokens = [&](const i32x4f_t& chunk, int (&cb)[NS]) {
        cnt = __builtin_amdgcn_readfirstlane(chunk[2]);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int j = chunk[1] + (s * 4 + r4 < cnt ? s * 4 + r4 : 0);
            row_of[s] = moe ? list.pair[j] : j;
            const int t = moe ? list.token[j] : j;
            cb[s] = t * pitch;  // the codes open few_lds
            xs[s] = scale[t];
        }
    };
    auto done = [&](int it, int (&sum)[NS], const f32x2v_t& sc) {
        const int i = 2 * it + o;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            uint32_t g = (uint32_t)sum[s], u = g;  // lanes 0..: gate of output 0, 16..: its up, 32.., 48..: of output 1
            swap16(g, u);
            const uint16_t v = f32_to_h<T>(gated((int)g, (int)u, xs[s], sc[0], sc[1], p.act));
            if ((lane & 31) < 4 && i < I && s * 4 + r4 < cnt) p.y[row_of[s] * p.ldy + i] = v;
        }
    };
    work.run(ring, wv, p.K, slots, enter, row, scales, tokens, done);
    w4_lds_barrier();
    work.close(wv, slots, enter, scales, tokens, done);
}

struct FewDownParams {
    const uint16_t* h;                              // quantise: [P][I]
    const int8_t* hq; const float* hs;              // staged: codes [P][I], scales
    const FewList* list;                            // staged: in chunks of at most `rows` pairs
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
template <int T, int SRC, int NS, int D>
__global__ __launch_bounds__(kFewThreads, 2) void few_down_kernel(const FewDownParams p) {
    extern __shared__ __align__(16) uint8_t few_lds[];  // sums [block][P][4], then codes [rows][pitch]
    __shared__ __align__(16) FewList list;
    __shared__ __align__(16) FewListTemp temp;
    __shared__ __align__(16) FewSlots slots;
    __shared__ float scale[kFewPairs];
    __shared__ uint32_t mag[kFewPairs];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int npairs = p.M * p.topk, pitch = few_pitch(p.I, D);
    float* sums = (float*)few_lds;
    const int codes_at = p.block * npairs * 16;
    int8_t* codes = (int8_t*)few_lds + codes_at;
    FewQuantiser<T> quant(p.h, p.I, SRC == kFewQuantise ? npairs : 0, p.I);
    few_clear(slots);
    few_sid(temp, npairs, p.ids, p.E);
    if constexpr (SRC == kFewQuantise) {
        if (tid < kFewPairs) mag[tid] = 0;
        w4_lds_barrier();
        few_list(list, temp, npairs, p.topk, 4 * NS);
    } else {
        few_copy_list(list, p.list);
        w4_lds_barrier();
    }
    const int chunks = __builtin_amdgcn_readfirstlane(list.chunks), all_pairs = __builtin_amdgcn_readfirstlane(list.pairs);
    const int groups = (int)(p.H / 4);
    FewWork<NS, D> work;
    int g0, g1;
    few_share(groups, blockIdx.x, gridDim.x, g0, g1);
    g1 += g0;
    const int r4 = lane & 3;
    // the block of row groups, and the batch of chunks [c0, c1) with pairs from list.pair[base], that are worked on
    int gb = g0, nb = 0, c0 = 0, c1 = 0, base = 0, pairs = 0;
    const int8_t* w = nullptr;
    const float* ws = nullptr;
    auto row = [&](int it) { return w + (uint64_t)(uint32_t)(4 * it) * (uint32_t)p.ldw; };
    auto scales = [&](int it) { return f32x2v_t{ws[4 * it], 0.f}; };
    auto enter = [&](int c) {
        const i32x4f_t h = c1 > c0 ? list.chunk[c0 + c] : i32x4f_t{0, 0, 0, 0};
        const int e = __builtin_amdgcn_readfirstlane(h[0]);
        w = p.w + ((int64_t)e * p.H + 4 * gb + r4) * p.ldw;
        ws = p.ws + (int64_t)e * p.H + 4 * gb + few_row(lane);
        return h;
    };
    FewRing<D> ring;
    auto open_batch = [&](bool restage) {  // from chunk c0: its codes are copied and its first weights requested
        nb = g1 - gb < p.block ? g1 - gb : p.block;
        c1 = c0;
        base = c0 < chunks ? __builtin_amdgcn_readfirstlane(list.chunk[c0][1]) : 0;
        pairs = all_pairs;
        if (all_pairs <= p.rows) {
            c1 = chunks;
        } else {  // as many chunks as LDS holds the pairs of: 64 at a time
            pairs = 0;
            for (;;) {
                const int c = c1 + lane;
                const i32x4f_t h = list.chunk[c < kFewPairs ? c : 0];
                const uint64_t in = __ballot(c < chunks && h[1] + h[2] - base <= p.rows);
                const int n = in == ~0ull ? 64 : __builtin_ctzll(~in);  // places ascend: the first ones
                c1 += n;
                if (n < 64) break;
            }
            if (c1 > c0) pairs = __builtin_amdgcn_readfirstlane(list.chunk[c1 - 1][1] + list.chunk[c1 - 1][2]) - base;
        }
        work.per = nb;
        if (SRC == kFewStaged && restage) stage_codes(p.hq, p.I, list.pair + base, pairs, p.I, pitch, codes);
        work.prime(ring, 0, (c1 - c0) * nb, wv, p.I, enter, row, scales);
    };
    if constexpr (SRC == kFewStaged)
        if (tid < npairs && temp.sid[tid] >= 0) scale[tid] = p.hs[tid];
    open_batch(true);
    if constexpr (SRC == kFewQuantise) {
        quant.maxima(mag);
        w4_lds_barrier();
        quant.codes(mag, codes, scale, pitch);
        w4_lds_barrier();
    } else {
        few_staged_barrier<D>();
    }
    int pair[NS], cnt = 0;
    float hs[NS];
    auto tokens = [&](const i32x4f_t& chunk, int (&cb)[NS]) {
        cnt = __builtin_amdgcn_readfirstlane(chunk[2]);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int j = chunk[1] + (s * 4 + r4 < cnt ? s * 4 + r4 : 0);
            pair[s] = list.pair[j];
            hs[s] = scale[pair[s]];
            cb[s] = codes_at + (SRC == kFewQuantise ? pair[s] : j - base) * pitch;
        }
    };
    auto done = [&](int it, int (&sum)[NS], const f32x2v_t& sc) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
            if ((lane & 15) < 4 && s * 4 + r4 < cnt)
                sums[(it * npairs + pair[s]) * 4 + few_row(lane)] = ((float)sum[s] * hs[s]) * sc[0];
    };
    for (;;) {
        work.run(ring, wv, p.I, slots, enter, row, scales, tokens, done);
        w4_lds_barrier();  // everyone is done with the codes
        work.close(wv, slots, enter, scales, tokens, done);
        const int gs = gb, ns = nb;
        const bool more = c1 < chunks, restage = more || c0 > 0;  // chunks of this block
        c0 = more ? c1 : 0;
        gb = more ? gb : gb + nb;
        const bool last = gb >= g1;
        if (!last) open_batch(restage);  // its first weights travel while the sums are joined
        w4_lds_barrier();  // the batch's sums are there
        few_clear(slots);
        if (!more)
            for (int i = tid; i < p.M * ns * 4; i += kFewThreads) {
                const int t = few_div(i, ns * 4, __builtin_amdgcn_rcpf((float)(ns * 4))), r = i - t * ns * 4;  // r: row of the block
                float sum = 0.f;
                for (int j = 0; j < p.topk; ++j) {
                    const int q = t * p.topk + j;
                    if (temp.sid[q] >= 0) sum = fmaf(p.gw[q], sums[((r >> 2) * npairs + q) * 4 + (r & 3)], sum);
                }
                p.y[t * p.ldy + 4 * gs + r] = f32_to_h<T>(sum);
            }
        if (last) break;
        few_staged_barrier<0>();
    }
}

}  // namespace qlin
