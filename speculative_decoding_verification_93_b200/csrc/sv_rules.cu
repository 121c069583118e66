// sv_rules.cu -- per-request rules on block logits: penalties for repeated
// tokens, biases, grammar masks (the formulas stand at sv_logits_process in
// include/sv.h).
//
// The rules change few logits: the tokens a request has seen (a few thousand
// of 129280), its biased tokens, and what its grammar forbids.  So nothing
// walks the vocabulary rule by rule.  One CTA takes a chunk of one row's
// vocabulary and every scheduled position of that chunk:
//   A. the chunk's bit planes (prompt, output; drafts and biases are OR-ed
//      in) are read once, V / 8 bytes each, and compacted into a list of the
//      touched tokens in shared memory;
//   B. in place, 16-byte units of the masked positions: units a mask forbids
//      whole are overwritten without being read, mixed ones written element by
//      element; with a separate output every unit is copied, masked on the way;
//   C. the touched tokens: in place a thread takes up to four positions of a
//      token, whose logits and mask words are requested together with the
//      token's count; with a separate output a (token, position) each, after
//      that position's copy, while its lines are still in the caches.
//      (Penalising inside the copy was slower, 66 against 59 us at
//      64 x 5 x 129280 bf16: a few lanes of a warp had work.)
//   D. the chunk's biased tokens, in place as further items of C; where a chunk
//      has more than a CTA lists, token by token.  Either way a token's last entry
//      is found once, and a list costs its length in every CTA of its row.
// In place, B and C/D touch disjoint elements (forbidden, allowed).
//
// Measured, bf16, 256 x 9 x 129280 in place, 1214 positions scheduled, 1.9 M
// touched logits, a quarter of the rows masked: 80 us on fresh logits, 74 on the
// same ones again, of which penalties alone take 39, masks alone 30 and a call
// without rules 9.  Slots and a status word add less than 2.  Touched logits lie alone
// in their sectors, so the DRAM moves 178 MB for the 66 MB that the rules name;
// it is a third busy, the issue slots half: the rest is waiting for a few
// logits at a time, CTA by CTA, six resident or five alike.
// 64 x 5 x 129280 with a separate output: 54 us, 36 of them the copy (165 MB,
// 4.6 TB/s); 128 x 17 x 129280 fp32, half of it scheduled: 240 us, 195 of them
// the copy (1.2 GB, 6.1 TB/s).
#include <climits>
#include <cstdint>

#include "sv.h"
#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

constexpr int kBiasList = 256;           // biases of a chunk that a CTA lists

// In place a CTA mostly waits (for its row's parameters, its planes, then a few
// logits each), so it takes many tokens; a copy is bound by its bytes, and small
// CTAs keep more of them on their way.  At the size above, in place on the same
// logits again: 8192 tokens and 256 threads 74 us; chunks of 4096 tokens 91, 128
// threads a CTA 93, 512 threads 112, chunks that grow with the token id 79.
template <bool IN_PLACE> struct RuleCfg {
    static constexpr int kThreads = IN_PLACE ? 256 : 128;
    static constexpr int kPlane = IN_PLACE ? kThreads : kThreads / 2;   // words of a plane
    static constexpr int kChunk = 32 * kPlane;           // tokens
    static constexpr int kResident = IN_PLACE ? 5 : 8;   // CTAs on an SM
};

struct RuleArgs {
    const char *in;
    char *out;
    int B, P, V, v0, Vs, W, nchunk;
    const int32_t *drafts;
    int K, pos0;
    const int32_t *lengths;
    int extra;
    const uint32_t *prompt, *output;   // null: empty history
    const int32_t *counts;
    int R;
    const int32_t *slots;
    const float *rep, *freq, *pres;
    const int32_t *bias_begin, *bias_tokens;
    const float *bias_values;
    int n_bias;
    const uint32_t *mask;
    int n_masks;
    const int32_t *mask_index;
    int32_t *status;
};

// 32 bits of a plane of W words from bit v on (bits past the plane are 0).
__device__ __forceinline__ uint32_t bits32(const uint32_t *plane, int W, int v) {
    const int w = v >> 5, s = v & 31;
    const uint32_t lo = w < W ? __ldg(plane + w) : 0u;
    if (s == 0) return lo;
    const uint32_t hi = w + 1 < W ? __ldg(plane + w + 1) : 0u;
    return __funnelshift_r(lo, hi, s);
}

// The bits of a logit, to be widened once every load of a batch is out: a
// conversion right behind its load would wait for it.
template <int ESIZE> __device__ __forceinline__ uint32_t ld_raw(const char *p) {
    if (ESIZE == 4) return *reinterpret_cast<const uint32_t *>(p);
    return *reinterpret_cast<const unsigned short *>(p);
}
template <int ESIZE> __device__ __forceinline__ float widen(uint32_t raw) {
    return __uint_as_float(ESIZE == 4 ? raw : raw << 16);
}

template <int ESIZE> __device__ __forceinline__ void st_logit(char *p, float z) {
    if (ESIZE == 4) *reinterpret_cast<float *>(p) = z;
    else *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(z);
}

template <bool IN_PLACE> struct RuleSmem {
    using Cfg = RuleCfg<IN_PLACE>;
    uint32_t draft[Cfg::kPlane];     // planes of the chunk, bit = local token
    uint32_t bias[Cfg::kPlane];
    uint32_t prompt[Cfg::kPlane];
    uint32_t output[Cfg::kPlane];
    alignas(4) unsigned short list[Cfg::kChunk];   // touched tokens without a bias, ascending
    int count[IN_PLACE ? 1 : Cfg::kChunk];   // output count of each listed token
    // More than kBiasList biases: the last entry of each of kLast tokens, where
    // the list (the counts) stood.
    static constexpr int kLast = IN_PLACE ? Cfg::kChunk / 2 : Cfg::kChunk;
    __device__ __forceinline__ int *last() { return IN_PLACE ? reinterpret_cast<int *>(list) : count; }
    int wsum[Cfg::kThreads / 32];
    int nbias;                       // valid biases of this chunk, and the first of them:
    int blist[kBiasList];            //   entry
    unsigned short btoken[kBiasList];   //   local token
    float bvalue[kBiasList];         //   value; NaN where a later entry counts
    int dup;                         // a biased token of this chunk is listed twice
    int dtok[SV_MAX_K];              // local token of each draft, -1 if not in the chunk
    int mask[SV_MAX_K + 1];          // mask of each position, -1 for none
};

struct RowRules {
    float rep, freq, pres;
    int slot;                        // -1: empty history
};

// Status bits of a row's own parameters; the invalid ones become neutral.
__device__ __forceinline__ int row_rules(const RuleArgs &a, int b, RowRules *r) {
    int bits = 0;
    r->rep = a.rep ? __ldg(a.rep + b) : 1.f;
    r->freq = a.freq ? __ldg(a.freq + b) : 0.f;
    r->pres = a.pres ? __ldg(a.pres + b) : 0.f;
    r->slot = -1;
    if (a.prompt) {
        r->slot = a.slots ? __ldg(a.slots + b) : b;
        if (r->slot < 0 || r->slot >= a.R) { r->slot = -1; bits |= SV_ROW_BAD_SLOT; }
    }
    if (!(r->rep > 0.f) || isinf(r->rep)) { r->rep = 1.f; bits |= SV_ROW_BAD_PENALTY; }
    if (!isfinite(r->freq)) { r->freq = 0.f; bits |= SV_ROW_BAD_PENALTY; }
    if (!isfinite(r->pres)) { r->pres = 0.f; bits |= SV_ROW_BAD_PENALTY; }
    return bits;
}

__device__ __forceinline__ const uint32_t *mask_row(const RuleArgs &a, int m) {
    return m < 0 ? nullptr : a.mask + static_cast<long long>(m) * a.W;
}

__device__ __forceinline__ bool allowed(const uint32_t *mask, int v) {
    return !mask || (__ldg(mask + (v >> 5)) >> (v & 31) & 1u);
}

// Output count of token lv of the chunk at c0.
template <bool IN_PLACE>
__device__ __forceinline__ int output_count(const RuleArgs &a, const RowRules &r, const RuleSmem<IN_PLACE> &sm,
                                            int c0, int lv) {
    return sm.output[lv >> 5] >> (lv & 31) & 1u
               ? __ldg(a.counts + static_cast<long long>(r.slot) * a.V + a.v0 + c0 + lv) : 0;
}

// Penalties of token lv at position p, on logit z; c: its output count.
template <bool IN_PLACE>
__device__ __forceinline__ float penalise(const RuleArgs &a, const RowRules &r, const RuleSmem<IN_PLACE> &sm,
                                          int lv, int c, int p, int ndraft, float z) {
    const uint32_t bit = 1u << (lv & 31);
    if (sm.draft[lv >> 5] & bit) {
        const int before = min(a.pos0 + p, ndraft);
        for (int j = 0; j < before; ++j) c += sm.dtok[j] == lv;
    }
    if (c > 0 || (sm.prompt[lv >> 5] & bit)) z = z > 0.f ? z / r.rep : z * r.rep;
    z -= r.freq * static_cast<float>(c);
    if (c > 0) z -= r.pres;
    return z;
}

// -inf wherever `keep` (one bit per element) is 0.
template <int ESIZE> __device__ __forceinline__ uint4 mask_unit(uint4 u, uint32_t keep) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (ESIZE == 4) {
            if (!(keep >> q & 1u)) w[q] = 0xff800000u;
        } else {
            if (!(keep >> (2 * q) & 1u)) w[q] = (w[q] & 0xffff0000u) | 0xff80u;
            if (!(keep >> (2 * q + 1) & 1u)) w[q] = (w[q] & 0x0000ffffu) | 0xff800000u;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// N bits of a mask from token v on, a second word only where they need one.
template <int N> __device__ __forceinline__ uint32_t mask_bits(const uint32_t *mask, int W, int v) {
    const int w = v >> 5, s = v & 31;
    uint32_t bits = __ldg(mask + w) >> s;
    if (s + N > 32 && w + 1 < W) bits |= __ldg(mask + w + 1) << (32 - s);
    return bits & ((1u << N) - 1u);
}

// The 16-byte units u0 .. u1 - 1 of a vector's elements c0 .. c0 + n - 1 (unit u
// starts at element head + kPer u), and the single elements beside them:
// [c0, first) and [last, c0 + n).
struct Units {
    int head, u0, u1, first, last;
};

template <int ESIZE> __device__ __forceinline__ Units units_of(const char *vec, int c0, int n, bool any) {
    constexpr int kPer = 16 / ESIZE;
    Units s;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(vec) & 15u);
    s.head = mis ? (16 - mis) / ESIZE : 0;
    s.u0 = s.u1 = 0;
    s.first = s.last = c0 + n;
    if (any) {
        s.u0 = c0 <= s.head ? 0 : (c0 - s.head + kPer - 1) / kPer;
        s.u1 = c0 + n <= s.head ? 0 : (c0 + n - s.head) / kPer;
        if (s.u1 > s.u0) { s.first = s.head + kPer * s.u0; s.last = s.head + kPer * s.u1; }
    }
    return s;
}

// B in place: -inf wherever a mask forbids.  A warp takes 128 units: each lane
// reads one word of the mask (of four positions at a time, so that a chunk's
// masks cost one or two round trips) and hands its units' bits round.
template <int ESIZE>
__device__ __forceinline__ void forbid(const RuleArgs &a, const RuleSmem<true> &sm, int b, int np, int c0, int n) {
    constexpr int kPer = 16 / ESIZE, kAhead = 4, kSpan = 128, kWords = kSpan * kPer / 32, kUnits = 32 / kPer;
    constexpr uint32_t kAll = (1u << kPer) - 1u;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const char *row = a.out + static_cast<long long>(b) * a.P * a.Vs * ESIZE;
    const long long vec = static_cast<long long>(a.Vs) * ESIZE;
    const int spans = (n / kPer + kSpan - 1) / kSpan;    // at most, whatever the alignment
    for (int span = warp; span < spans; span += RuleCfg<true>::kThreads / 32) {
        for (int p0 = 0; p0 < np; p0 += kAhead) {
            uint32_t w[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                w[k] = ~0u;
                const int m = p0 + k < np ? sm.mask[p0 + k] : -1;
                if (m >= 0 && lane < kWords) {
                    const Units s = units_of<ESIZE>(row + (p0 + k) * vec, c0, n, true);
                    const int v = a.v0 + s.head + kPer * (s.u0 + span * kSpan) + 32 * lane;
                    w[k] = bits32(a.mask + static_cast<long long>(m) * a.W, a.W, v);
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (p0 + k >= np || sm.mask[p0 + k] < 0) continue;
                const Units s = units_of<ESIZE>(row + (p0 + k) * vec, c0, n, true);
#pragma unroll
                for (int i = 0; i < kSpan / 32; ++i) {
                    const int u = s.u0 + span * kSpan + 32 * i + lane;
                    const uint32_t keep =
                        __shfl_sync(0xffffffffu, w[k], (32 * i + lane) / kUnits) >> (lane % kUnits * kPer) & kAll;
                    char *d = const_cast<char *>(row) + (p0 + k) * vec + static_cast<long long>(s.head + kPer * u) * ESIZE;
                    if (u >= s.u1) continue;
                    if (keep == 0) {
                        *reinterpret_cast<uint4 *>(d) = mask_unit<ESIZE>(make_uint4(0, 0, 0, 0), 0);
                    } else {
                        for (uint32_t f = keep ^ kAll; f; f &= f - 1) st_logit<ESIZE>(d + (__ffs(f) - 1) * ESIZE, kNegInf);
                    }
                }
            }
        }
    }
    // The elements before the first unit and behind the last.
    for (int q = tid; q < np * 2 * kPer; q += RuleCfg<true>::kThreads) {
        const int p = q / (2 * kPer), i = q % (2 * kPer);
        if (sm.mask[p] < 0) continue;
        const Units s = units_of<ESIZE>(row + p * vec, c0, n, true);
        const int before = s.first - c0, v = i < before ? c0 + i : s.last + i - before;
        if (v < c0 + n && !allowed(mask_row(a, sm.mask[p]), a.v0 + v))
            st_logit<ESIZE>(const_cast<char *>(row) + p * vec + static_cast<long long>(v) * ESIZE, kNegInf);
    }
}

// B with a separate output: position p of the chunk, copied and masked.
template <int ESIZE, bool MASKED>
__device__ __forceinline__ void copy_position(const RuleArgs &a, int b, int p, int c0, int n, const uint32_t *mask) {
    constexpr int kPer = 16 / ESIZE, kBatch = 4;
    constexpr uint32_t kAll = (1u << kPer) - 1u;
    const int tid = threadIdx.x;
    const long long vec = (static_cast<long long>(b) * a.P + p) * a.Vs;
    const char *src = a.in + vec * ESIZE;
    char *dst = a.out + vec * ESIZE;
    const Units s = units_of<ESIZE>(dst, c0, n, ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15u) == 0);
    // kBatch units a thread: all their loads before the first store.
    for (int base = s.u0 + tid; base < s.u1; base += kBatch * RuleCfg<false>::kThreads) {
        uint32_t keep[kBatch];
        uint4 data[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int u = base + k * RuleCfg<false>::kThreads;
            keep[k] = kAll;
            if (u < s.u1) {
                data[k] = ld_stream(src + static_cast<long long>(s.head + kPer * u) * ESIZE);
                if (MASKED) keep[k] = mask_bits<kPer>(mask, a.W, a.v0 + s.head + kPer * u);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int u = base + k * RuleCfg<false>::kThreads;
            if (u < s.u1)
                *reinterpret_cast<uint4 *>(dst + static_cast<long long>(s.head + kPer * u) * ESIZE) =
                    MASKED ? mask_unit<ESIZE>(data[k], keep[k]) : data[k];
        }
    }
    const int nscalar = (s.first - c0) + (c0 + n - s.last);
    for (int q = tid; q < nscalar; q += RuleCfg<false>::kThreads) {
        const int v = q < s.first - c0 ? c0 + q : s.last + (q - (s.first - c0));
        if (MASKED && !allowed(mask, a.v0 + v)) {
            st_logit<ESIZE>(dst + static_cast<long long>(v) * ESIZE, kNegInf);
        } else {                         // bits, not numbers: NaN payloads stay
            if (ESIZE == 4) reinterpret_cast<uint32_t *>(dst)[v] = reinterpret_cast<const uint32_t *>(src)[v];
            else reinterpret_cast<unsigned short *>(dst)[v] = reinterpret_cast<const unsigned short *>(src)[v];
        }
    }
}

__device__ __forceinline__ bool valid_bias(float v) { return !isnan(v) && !(isinf(v) && v > 0.f); }

// A ban gives -inf whatever the logit was: the sum of +inf or NaN with it is NaN.
__device__ __forceinline__ float biased(float z, float v) { return v == kNegInf ? kNegInf : z + v; }

// Of a token listed twice the later entry counts: the others' values become NaN.
template <bool IN_PLACE> __device__ __forceinline__ void drop_replaced(RuleSmem<IN_PLACE> &sm) {
    for (int i = threadIdx.x; i < sm.nbias; i += RuleCfg<IN_PLACE>::kThreads) {
        bool replaced = false;
        for (int j = 0; j < sm.nbias; ++j) replaced |= sm.btoken[j] == sm.btoken[i] && sm.blist[j] > sm.blist[i];
        if (replaced) sm.bvalue[i] = __builtin_nanf("");
    }
}

// Status: the row's parameters, and masks of its first np positions that allow
// nothing (a row's CTAs share them).
template <bool IN_PLACE>
__device__ __forceinline__ void report(const RuleArgs &a, const RuleSmem<IN_PLACE> &sm, int chunk, int np, int bits) {
    if (!a.status) return;
    for (int p = chunk; p < np; p += a.nchunk) {
        const uint32_t *mask = mask_row(a, sm.mask[p]);
        if (!mask) continue;
        uint32_t any = 0;
        for (int w = threadIdx.x; w < a.W && !any; w += RuleCfg<IN_PLACE>::kThreads) {
            any = __ldg(mask + w);
            if (w == a.W - 1 && (a.V & 31)) any &= (1u << (a.V & 31)) - 1u;
        }
        if (!__syncthreads_or(any != 0) && threadIdx.x == 0) bits |= SV_ROW_EMPTY_MASK;
    }
    if (bits) atomicOr(a.status, bits);
}

template <int ESIZE, bool IN_PLACE>
__global__ void __launch_bounds__(RuleCfg<IN_PLACE>::kThreads, RuleCfg<IN_PLACE>::kResident) rules_kernel(RuleArgs a) {
    using Cfg = RuleCfg<IN_PLACE>;
    __shared__ RuleSmem<IN_PLACE> sm;
    constexpr int kThreads = Cfg::kThreads;
    constexpr int kTokens = 2;           // touched tokens on their way at a time (copy)
    constexpr int kPositions = 4;        // positions of a touched token on their way at a time (in place)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Rows fastest: the low chunks, where most of a text's tokens lie, first.
    const int chunk = blockIdx.x / a.B, b = blockIdx.x - chunk * a.B;
    const int c0 = chunk * Cfg::kChunk, n = min(Cfg::kChunk, a.Vs - c0);
    griddep_wait();
    griddep_launch_dependents();

    // Everything about the row in one round trip, its planes too where its slot
    // needs no lookup.
    uint32_t wp = 0, wo = 0;
    auto planes = [&](int slot) {
        const long long row = static_cast<long long>(slot) * a.W;
        wo = bits32(a.output + row, a.W, a.v0 + c0 + 32 * tid);
        wp = bits32(a.prompt + row, a.W, a.v0 + c0 + 32 * tid);
    };
    if (a.prompt && !a.slots && 32 * tid < n) planes(b);
    const int len = a.lengths ? __ldg(a.lengths + b) : 0;
    RowRules r;
    int bits = row_rules(a, b, &r);
    int e0 = 0, e1 = 0;
    if (a.bias_begin) {
        e0 = __ldg(a.bias_begin + b);
        e1 = __ldg(a.bias_begin + b + 1);
        if (e0 < 0 || e1 < e0 || e1 > a.n_bias) { e0 = e1 = 0; bits |= SV_ROW_BAD_BIAS; }
    }
    const int x = tid < a.K ? __ldg(a.drafts + static_cast<long long>(b) * a.K + tid) : 0;
    int m = -1;
    if (a.mask && tid < a.P) {
        const long long q = static_cast<long long>(b) * a.P + tid;
        m = a.mask_index ? __ldg(a.mask_index + q) : static_cast<int>(q);
    }
    // Scheduled positions of this row among the P given.
    long long np_l = a.P;
    if (a.lengths) np_l = static_cast<long long>(len) + a.extra - a.pos0;
    const int np = static_cast<int>(max(0ll, min(np_l, static_cast<long long>(a.P))));
    if (np == 0) return;
    if (m < -1 || m >= a.n_masks) {
        m = -1;
        if (tid < np) bits |= SV_ROW_BAD_MASK;
    }
    const bool penal = r.rep != 1.f || r.freq != 0.f || r.pres != 0.f;
    const int ndraft = min(a.K, a.pos0 + np - 1);   // drafts before the last position
    if (tid < ndraft && (x < 0 || x >= a.V)) bits |= SV_ROW_BAD_TOKEN;
    if (tid <= SV_MAX_K) sm.mask[tid] = m;
    if (tid == 0) sm.dup = sm.nbias = 0;
    for (int w = tid; w < Cfg::kPlane; w += kThreads) sm.draft[w] = sm.bias[w] = 0;
    // The bias list's first entries are on their way over the barrier.
    if (penal && a.slots && r.slot >= 0 && 32 * tid < n) planes(r.slot);
    int bt = -1;
    float bv = 0.f;
    if (e0 + tid < e1) {
        bt = __ldg(a.bias_tokens + e0 + tid);
        bv = __ldg(a.bias_values + e0 + tid);
    }
    const bool masked = __syncthreads_or(tid < np && m >= 0);
    if constexpr (IN_PLACE) {
        if (masked) forbid<ESIZE>(a, sm, b, np, c0, n);
        if (!penal && e0 == e1) {                         // no more rules
            report(a, sm, chunk, masked ? np : 0, bits);
            return;
        }
    }
    // A. Planes of the chunk, drafts and biases.
    if (tid < ndraft) {
        int lv = -1;
        if (x >= 0 && x < a.V && x >= a.v0 + c0 && x < a.v0 + c0 + n) lv = x - a.v0 - c0;
        sm.dtok[tid] = lv;
        if (lv >= 0 && penal) atomicOr(&sm.draft[lv >> 5], 1u << (lv & 31));
    }
    for (int e = e0 + tid; e < e1; e += kThreads) {
        if (e != e0 + tid) {
            bt = __ldg(a.bias_tokens + e);
            bv = __ldg(a.bias_values + e);
        }
        if (bt < 0 || bt >= a.V) { bits |= SV_ROW_BAD_TOKEN; continue; }
        if (!valid_bias(bv)) { bits |= SV_ROW_BAD_BIAS; continue; }
        const int lv = bt - a.v0 - c0;
        if (lv < 0 || lv >= n) continue;
        const uint32_t bit = 1u << (lv & 31);
        if (atomicOr(&sm.bias[lv >> 5], bit) & bit) sm.dup = 1;
        const int i = atomicAdd(&sm.nbias, 1);
        if (i < kBiasList) {
            sm.blist[i] = e;
            sm.btoken[i] = static_cast<unsigned short>(lv);
            sm.bvalue[i] = bv;
        }
    }
    const uint32_t live = !penal || n <= 32 * tid ? 0u : n - 32 * tid >= 32 ? ~0u : (1u << (n - 32 * tid)) - 1u;
    wo &= live;
    wp &= r.rep != 1.f ? live : 0u;
    if (tid < Cfg::kPlane) {
        sm.prompt[tid] = wp;
        sm.output[tid] = wo;
    }
    __syncthreads();
    if (sm.dup && sm.nbias <= kBiasList) drop_replaced(sm);
    // The touched tokens in ascending order: places by a scan over the words.
    uint32_t touched = tid < Cfg::kPlane ? (wp | wo | sm.draft[tid]) & ~sm.bias[tid] : 0u;
    int incl = __popc(touched);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sm.wsum[warp] = incl;
    __syncthreads();
    int at = incl - __popc(touched), ntouched = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += sm.wsum[w];
        ntouched += sm.wsum[w];
    }
    for (; touched; touched &= touched - 1) sm.list[at++] = 32 * tid + __ffs(touched) - 1;
    __syncthreads();

    const long long vec = static_cast<long long>(a.Vs) * ESIZE;
    const long long row_at = (static_cast<long long>(b) * a.P * a.Vs + c0) * ESIZE;
    if (!IN_PLACE) {
        for (int q = tid; q < ntouched; q += kThreads) sm.count[q] = output_count(a, r, sm, c0, sm.list[q]);
        for (int p = 0; p < np; ++p) {
            const uint32_t *mask = mask_row(a, sm.mask[p]);
            const char *src = a.in + row_at + p * vec;
            char *dst = a.out + row_at + p * vec;
            // C's first logits are on their way during the copy.
            uint32_t z[kTokens], word[kTokens];
            auto ask = [&](int q0) {
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    const int q = q0 + k * kThreads, lv = q < ntouched ? sm.list[q] : 0;
                    z[k] = ld_raw<ESIZE>(src + lv * ESIZE);
                    word[k] = ~0u;
                    if (mask) word[k] = __ldg(mask + ((a.v0 + c0 + lv) >> 5));
                }
            };
            if (ntouched) ask(tid);
            if (mask) copy_position<ESIZE, true>(a, b, p, c0, n, mask);
            else copy_position<ESIZE, false>(a, b, p, c0, n, nullptr);
            __syncthreads();
            for (int q0 = tid; q0 < ntouched; q0 += kTokens * kThreads) {
                if (q0 != tid) ask(q0);
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    const int q = q0 + k * kThreads;
                    if (q >= ntouched) break;
                    const int lv = sm.list[q];
                    if (word[k] >> ((a.v0 + c0 + lv) & 31) & 1u)
                        st_logit<ESIZE>(dst + lv * ESIZE,
                                        penalise(a, r, sm, lv, sm.count[q], p, ndraft, widen<ESIZE>(z[k])));
                }
            }
        }
        __syncthreads();
    } else {
        // C. Tokens fastest.  A forbidden logit is read too: waiting for its
        // mask first would cost a second round trip.
        // The biased tokens (D) come behind the touched ones in the same order,
        // so that theirs is not a round trip of its own.
        const int items = ntouched + (sm.nbias <= kBiasList ? sm.nbias : 0);
        if (items > 0) {
            const int units = (np + kPositions - 1) / kPositions;    // positions u, u + units, ... a thread
            const int dq = kThreads / items, dr = kThreads % items;
            int q = tid % items, u = tid / items;
            while (u < units) {
                const int bias = q - ntouched, lv = bias < 0 ? sm.list[q] : sm.btoken[bias];
                const long long at = row_at + lv * ESIZE;
                const int t = a.v0 + c0 + lv;
                uint32_t z[kPositions], word[kPositions];
#pragma unroll
                for (int k = 0; k < kPositions; ++k) {
                    const int p = u + k * units;
                    word[k] = ~0u;
                    if (p < np) {
                        z[k] = ld_raw<ESIZE>(a.in + at + p * vec);
                        if (masked)
                            if (const uint32_t *mask = mask_row(a, sm.mask[p])) word[k] = __ldg(mask + (t >> 5));
                    }
                }
                const int c = output_count(a, r, sm, c0, lv);
                const float more = bias >= 0 ? sm.bvalue[bias] : 0.f;
#pragma unroll
                for (int k = 0; k < kPositions; ++k) {
                    const int p = u + k * units;
                    if (p >= np || !(word[k] >> (t & 31) & 1u) || isnan(more)) continue;
                    float y = penalise(a, r, sm, lv, c, p, ndraft, widen<ESIZE>(z[k]));
                    if (bias >= 0) y = biased(y, more);
                    st_logit<ESIZE>(a.out + at + p * vec, y);
                }
                q += dr;
                u += dq;
                if (q >= items) { q -= items; ++u; }
            }
        }
    }
    // D. Biased tokens.  Position p of token lv, with bias v.
    auto bias_logit = [&](int lv, int p, int c, float v) {
        const long long to = row_at + p * vec + lv * ESIZE;
        const uint32_t raw = ld_raw<ESIZE>(a.in + to);
        if (!allowed(mask_row(a, sm.mask[p]), a.v0 + c0 + lv)) return;
        float z = widen<ESIZE>(raw);
        if (penal) z = penalise(a, r, sm, lv, c, p, ndraft, z);
        st_logit<ESIZE>(a.out + to, biased(z, v));
    };
    if (sm.nbias > kBiasList) {
        for (int l0 = 0; l0 < n; l0 += sm.kLast) {
            const int m = min(sm.kLast, n - l0);
            __syncthreads();                  // what stood there has been read
            for (int lv = tid; lv < m; lv += kThreads) sm.last()[lv] = -1;
            __syncthreads();
            for (int e = e0 + tid; e < e1; e += kThreads) {
                const int t = __ldg(a.bias_tokens + e);
                if (t < 0 || t >= a.V || !valid_bias(__ldg(a.bias_values + e))) continue;
                const int lv = t - a.v0 - c0 - l0;
                if (lv >= 0 && lv < m) atomicMax(&sm.last()[lv], e);
            }
            __syncthreads();
            for (int lv = tid; lv < m; lv += kThreads) {
                const int e = sm.last()[lv];
                if (e < 0) continue;
                const float v = __ldg(a.bias_values + e);
                const int c = penal ? output_count(a, r, sm, c0, l0 + lv) : 0;
                for (int p = 0; p < np; ++p) bias_logit(l0 + lv, p, c, v);
            }
        }
    } else if (!IN_PLACE) {
        for (int q = tid; q < sm.nbias * np; q += kThreads) {
            const int i = q / np, lv = sm.btoken[i];
            const float v = sm.bvalue[i];
            if (!isnan(v)) bias_logit(lv, q - i * np, penal ? output_count(a, r, sm, c0, lv) : 0, v);
        }
    }

    report(a, sm, chunk, masked ? np : 0, bits);
}

}  // namespace sv

extern "C" sv_status sv_logits_process(const void *logits, void *out, sv_dtype dtype, int B, int P,
                                       int V, int v0, int Vs, const int32_t *draft_tokens, int K,
                                       int pos0, const int32_t *lengths, int extra,
                                       const sv_logit_rules *rules, int32_t *status, void *stream) {
    sv::NvtxRange nvtx_range("sv_logits_process");
    if (!rules) return SV_ERR_ARG;
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
    if (B < 0 || P < 1 || P > SV_MAX_K + 1 || V < 1 || V > SV_MAX_V || v0 < 0 || Vs < 1 ||
        Vs > V - v0 || K < 0 || K > SV_MAX_K || pos0 < 0 || pos0 > SV_MAX_K)
        return SV_ERR_SHAPE;
    if (B == 0) return SV_OK;
    if (!logits || !out || (K > 0 && !draft_tokens)) return SV_ERR_ARG;
    const size_t es = dtype == SV_F32 ? 4 : 2;
    const uintptr_t in_at = reinterpret_cast<uintptr_t>(logits), out_at = reinterpret_cast<uintptr_t>(out);
    if ((in_at | out_at) & (es - 1)) return SV_ERR_ARG;
    const size_t bytes = static_cast<size_t>(B) * P * Vs * es;
    if (in_at != out_at && in_at < out_at + bytes && out_at < in_at + bytes) return SV_ERR_ARG;
    if (sv::misaligned4(draft_tokens, lengths, status, rules->slots, rules->repetition, rules->frequency,
                        rules->presence, rules->bias_begin, rules->bias_tokens, rules->bias_values, rules->mask,
                        rules->mask_index))
        return SV_ERR_ARG;
    sv::RuleArgs a = {};
    if (const sv_history *h = rules->history) {
        if (!h->prompt_bits || !h->output_bits || !h->output_counts ||
            sv::misaligned4(h->prompt_bits, h->output_bits, h->output_counts))
            return SV_ERR_ARG;
        if (h->R < 1 || h->V != V || (!rules->slots && B > h->R)) return SV_ERR_SHAPE;
        a.prompt = h->prompt_bits;
        a.output = h->output_bits;
        a.counts = h->output_counts;
        a.R = h->R;
    }
    if (rules->bias_begin && (rules->n_bias < 0 ||
                              (rules->n_bias > 0 && (!rules->bias_tokens || !rules->bias_values))))
        return SV_ERR_ARG;
    if (rules->bias_begin && rules->n_bias > (1 << 30)) return SV_ERR_SHAPE;   // entry + thread stays an int
    if (rules->mask) {
        if (rules->n_masks < 1) return SV_ERR_ARG;
        if (!rules->mask_index && static_cast<long long>(B) * P > rules->n_masks) return SV_ERR_SHAPE;
    }
    a.in = static_cast<const char *>(logits);
    a.out = static_cast<char *>(out);
    a.B = B; a.P = P; a.V = V; a.v0 = v0; a.Vs = Vs;
    a.W = (V + 31) / 32;
    const bool in_place = in_at == out_at;
    const int chunk = in_place ? sv::RuleCfg<true>::kChunk : sv::RuleCfg<false>::kChunk;
    a.nchunk = (Vs + chunk - 1) / chunk;
    a.drafts = K > 0 ? draft_tokens : nullptr;
    a.K = K; a.pos0 = pos0;
    a.lengths = lengths; a.extra = extra;
    a.slots = rules->slots;
    a.rep = rules->repetition; a.freq = rules->frequency; a.pres = rules->presence;
    a.bias_begin = rules->bias_begin;
    a.bias_tokens = rules->bias_tokens; a.bias_values = rules->bias_values;
    a.n_bias = rules->n_bias;
    a.mask = rules->mask; a.n_masks = rules->n_masks; a.mask_index = rules->mask_index;
    a.status = status;
    const long long grid = static_cast<long long>(B) * a.nchunk;
    if (grid > INT_MAX) return SV_ERR_SHAPE;
    auto *kernel = dtype == SV_F32 ? (in_place ? sv::rules_kernel<4, true> : sv::rules_kernel<4, false>)
                                   : (in_place ? sv::rules_kernel<2, true> : sv::rules_kernel<2, false>);
    return sv::note_cuda(sv::launch_pdl(kernel, dim3(static_cast<unsigned>(grid)),
                                        dim3(in_place ? sv::RuleCfg<true>::kThreads : sv::RuleCfg<false>::kThreads), 0,
                                        static_cast<cudaStream_t>(stream), a));
}
