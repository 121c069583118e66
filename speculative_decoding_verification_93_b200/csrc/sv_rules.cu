// sv_rules.cu -- per-request rules on block logits: penalties for repeated
// tokens, biases, grammar masks (the formulas stand at sv_logits_process in
// include/sv.h).
//
// The rules change few logits: the tokens a request has seen (a few thousand
// of 129280), its biased tokens, and what its grammar forbids.  So nothing
// walks the vocabulary logit by logit.  One CTA takes kChunk tokens of one
// row and every scheduled position of that chunk:
//   A. the chunk's bit planes (prompt, output; drafts and biases are OR-ed
//      in) are read once, V / 8 bytes each, and compacted into a list of the
//      touched tokens in shared memory;
//   B. per position, 16-byte units: in place, units whose mask byte forbids
//      all eight (fp32: four) logits are overwritten without being read, and
//      mixed units are written element by element; with a separate output
//      the unit is copied with the forbidden elements replaced;
//   C. (position, list entry) pairs over all threads: read the logit and its
//      count, apply the penalties, write;  D. the same for biased tokens.
// In place, B and C/D touch disjoint elements (forbidden, allowed); with a
// separate output a barrier orders them.
#include <climits>
#include <cstdint>

#include "sv.h"
#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

constexpr int kRuleThreads = 256;
constexpr int kChunk = 32 * kRuleThreads;   // tokens per CTA: one bit-plane word per thread

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

template <int ESIZE> __device__ __forceinline__ float ld_logit(const char *p) {
    if (ESIZE == 4) return *reinterpret_cast<const float *>(p);
    return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const unsigned short *>(p)) << 16);
}

template <int ESIZE> __device__ __forceinline__ void st_logit(char *p, float z) {
    if (ESIZE == 4) *reinterpret_cast<float *>(p) = z;
    else *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(z);
}

struct RuleSmem {
    uint32_t draft[kRuleThreads];    // planes of the chunk, bit = local token
    uint32_t bias[kRuleThreads];
    uint32_t prompt[kRuleThreads];
    uint32_t output[kRuleThreads];
    unsigned short list[kChunk];     // touched local tokens without a bias
    int n;
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

// What a token's history says: its count before the block, the prompt's bit,
// and whether the block's drafts name it.
struct TokenState {
    int count;
    bool prompt, draft;
};

__device__ __forceinline__ TokenState token_state(const RuleArgs &a, const RowRules &r, const RuleSmem &sm,
                                                  int c0, int lv) {
    const uint32_t bit = 1u << (lv & 31);
    TokenState s;
    s.count = 0;
    if (sm.output[lv >> 5] & bit)
        s.count = __ldg(a.counts + static_cast<long long>(r.slot) * a.V + a.v0 + c0 + lv);
    s.prompt = sm.prompt[lv >> 5] & bit;
    s.draft = sm.draft[lv >> 5] & bit;
    return s;
}

// Penalties of a token at position p, on logit z.
__device__ __forceinline__ float penalise(const RuleArgs &a, const RowRules &r, const RuleSmem &sm,
                                          const TokenState &s, int lv, int p, int ndraft, float z) {
    int c = s.count;
    if (s.draft) {
        const int before = min(a.pos0 + p, ndraft);
        for (int j = 0; j < before; ++j) c += sm.dtok[j] == lv;
    }
    if (c > 0 || s.prompt) z = z > 0.f ? z / r.rep : z * r.rep;
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

// B. Position p of the chunk: masks, and the copy when the output is separate.
template <int ESIZE, bool IN_PLACE, bool MASKED>
__device__ __forceinline__ void mask_position(const RuleArgs &a, int b, int p, int c0, int n, const uint32_t *mask) {
    constexpr int kPer = 16 / ESIZE, kBatch = 4;
    constexpr uint32_t kAll = (1u << kPer) - 1u;
    const int tid = threadIdx.x;
    const long long vec = (static_cast<long long>(b) * a.P + p) * a.Vs;
    const char *src = a.in + vec * ESIZE;
    char *dst = a.out + vec * ESIZE;
    // Units start at the elements head + kPer u of the vector.
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(dst) & 15u);
    const int head = mis ? (16 - mis) / ESIZE : 0;
    int u0 = 0, u1 = 0, first = c0 + n, last = c0 + n;   // single elements: [c0, first) and [last, c0 + n)
    if (IN_PLACE || ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15u) == 0) {
        u0 = c0 <= head ? 0 : (c0 - head + kPer - 1) / kPer;
        u1 = c0 + n <= head ? 0 : (c0 + n - head) / kPer;
        if (u1 > u0) { first = head + kPer * u0; last = head + kPer * u1; }
    }
    // kBatch units a thread: all their loads before the first store.
    for (int base = u0 + tid; base < u1; base += kBatch * kRuleThreads) {
        uint32_t keep[kBatch];
        uint4 data[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int u = base + k * kRuleThreads;
            keep[k] = kAll;
            if (u < u1) {
                if (!IN_PLACE) data[k] = ld_stream(src + static_cast<long long>(head + kPer * u) * ESIZE);
                if (MASKED) keep[k] = mask_bits<kPer>(mask, a.W, a.v0 + head + kPer * u);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int u = base + k * kRuleThreads;
            char *d = dst + static_cast<long long>(head + kPer * u) * ESIZE;
            if (u >= u1) continue;
            if (!IN_PLACE) {
                *reinterpret_cast<uint4 *>(d) = MASKED ? mask_unit<ESIZE>(data[k], keep[k]) : data[k];
            } else if (keep[k] == 0) {
                *reinterpret_cast<uint4 *>(d) = mask_unit<ESIZE>(make_uint4(0, 0, 0, 0), 0);
            } else {
                for (uint32_t m = keep[k] ^ kAll; m; m &= m - 1) st_logit<ESIZE>(d + (__ffs(m) - 1) * ESIZE, kNegInf);
            }
        }
    }
    const int nscalar = (first - c0) + (c0 + n - last);
    for (int q = tid; q < nscalar; q += kRuleThreads) {
        const int v = q < first - c0 ? c0 + q : last + (q - (first - c0));
        if (MASKED && !allowed(mask, a.v0 + v))
            st_logit<ESIZE>(dst + static_cast<long long>(v) * ESIZE, kNegInf);
        else if (!IN_PLACE)
            st_logit<ESIZE>(dst + static_cast<long long>(v) * ESIZE, ld_logit<ESIZE>(src + static_cast<long long>(v) * ESIZE));
    }
}

__device__ __forceinline__ bool valid_bias(float v) { return !isnan(v) && !(isinf(v) && v > 0.f); }

template <int ESIZE, bool IN_PLACE>
__global__ void __launch_bounds__(kRuleThreads) rules_kernel(RuleArgs a) {
    __shared__ RuleSmem sm;
    constexpr int kBatch = 4;
    const int tid = threadIdx.x;
    // Rows fastest: the low chunks, where most of a text's tokens lie, first.
    const int chunk = blockIdx.x / a.B, b = blockIdx.x - chunk * a.B;
    griddep_wait();
    griddep_launch_dependents();
    const int c0 = chunk * kChunk, n = min(kChunk, a.Vs - c0);

    // Everything about the row in one round trip.
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

    // A. Planes of the chunk, drafts and biases.
    uint32_t wp = 0, wo = 0;
    if (penal && r.slot >= 0 && 32 * tid < n) {
        const uint32_t live = n - 32 * tid >= 32 ? ~0u : (1u << (n - 32 * tid)) - 1u;
        const long long row = static_cast<long long>(r.slot) * a.W;
        wo = bits32(a.output + row, a.W, a.v0 + c0 + 32 * tid) & live;
        if (r.rep != 1.f) wp = bits32(a.prompt + row, a.W, a.v0 + c0 + 32 * tid) & live;
    }
    const int ndraft = min(a.K, a.pos0 + np - 1);   // drafts before the last position
    if (tid == 0) { sm.n = 0; sm.dup = 0; }
    if (tid <= SV_MAX_K) sm.mask[tid] = m;
    sm.draft[tid] = 0;
    sm.bias[tid] = 0;
    sm.prompt[tid] = wp;
    sm.output[tid] = wo;
    __syncthreads();
    if (tid < ndraft) {
        int lv = -1;
        if (x < 0 || x >= a.V) bits |= SV_ROW_BAD_TOKEN;
        else if (x >= a.v0 + c0 && x < a.v0 + c0 + n) lv = x - a.v0 - c0;
        sm.dtok[tid] = lv;
        if (lv >= 0 && penal) atomicOr(&sm.draft[lv >> 5], 1u << (lv & 31));
    }
    for (int e = e0 + tid; e < e1; e += kRuleThreads) {
        const int t = __ldg(a.bias_tokens + e);
        const float v = __ldg(a.bias_values + e);
        if (t < 0 || t >= a.V) { bits |= SV_ROW_BAD_TOKEN; continue; }
        if (!valid_bias(v)) { bits |= SV_ROW_BAD_BIAS; continue; }
        const int lv = t - a.v0 - c0;
        if (lv < 0 || lv >= n) continue;
        const uint32_t bit = 1u << (lv & 31);
        if (atomicOr(&sm.bias[lv >> 5], bit) & bit) sm.dup = 1;
    }
    __syncthreads();
    uint32_t touched = (wp | wo | sm.draft[tid]) & ~sm.bias[tid];
    if (touched) {
        int at = atomicAdd(&sm.n, __popc(touched));
        for (; touched; touched &= touched - 1) sm.list[at++] = 32 * tid + __ffs(touched) - 1;
    }

    // B. Masks, and the copy when the output is separate.
    for (int p = 0; p < np; ++p) {
        const uint32_t *mask = mask_row(a, sm.mask[p]);
        if (mask) mask_position<ESIZE, IN_PLACE, true>(a, b, p, c0, n, mask);
        else if (!IN_PLACE) mask_position<ESIZE, IN_PLACE, false>(a, b, p, c0, n, nullptr);
    }
    __syncthreads();

    // C. Penalised tokens without a bias: a token a thread, kBatch positions
    // on their way at a time.
    const long long row_at = (static_cast<long long>(b) * a.P * a.Vs + c0) * ESIZE;
    const long long vec = static_cast<long long>(a.Vs) * ESIZE;
    for (int q = tid; q < sm.n; q += kRuleThreads) {
        const int lv = sm.list[q];
        const TokenState s = token_state(a, r, sm, c0, lv);
        for (int p0 = 0; p0 < np; p0 += kBatch) {
            float z[kBatch];
            bool live[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int p = p0 + k;
                live[k] = p < np && allowed(mask_row(a, sm.mask[p]), a.v0 + c0 + lv);
                if (live[k]) z[k] = ld_logit<ESIZE>(a.in + row_at + p * vec + lv * ESIZE);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (live[k])
                    st_logit<ESIZE>(a.out + row_at + (p0 + k) * vec + lv * ESIZE,
                                    penalise(a, r, sm, s, lv, p0 + k, ndraft, z[k]));
        }
    }
    // D. Biased tokens: the last entry of a token counts.
    const long long pairs = static_cast<long long>(e1 - e0) * np;
    for (long long q = tid; q < pairs; q += kRuleThreads) {
        const int e = e0 + static_cast<int>(q / np), p = static_cast<int>(q % np);
        const int t = __ldg(a.bias_tokens + e), lv = t - a.v0 - c0;
        if (t < 0 || t >= a.V || lv < 0 || lv >= n) continue;
        const float v = __ldg(a.bias_values + e);
        if (!valid_bias(v)) continue;
        if (sm.dup) {
            bool later = false;
            for (int f = e + 1; f < e1 && !later; ++f)
                later = __ldg(a.bias_tokens + f) == t && valid_bias(__ldg(a.bias_values + f));
            if (later) continue;
        }
        if (!allowed(mask_row(a, sm.mask[p]), t)) continue;
        const long long at = row_at + p * vec + lv * ESIZE;
        float z = ld_logit<ESIZE>(a.in + at);
        if (penal) z = penalise(a, r, sm, token_state(a, r, sm, c0, lv), lv, p, ndraft, z);
        st_logit<ESIZE>(a.out + at, z + v);
    }

    // Status: the row's parameters, and masks that allow nothing (a row's
    // CTAs share its positions).
    if (!a.status) return;
    for (int p = chunk; p < np; p += a.nchunk) {
        const uint32_t *mask = mask_row(a, sm.mask[p]);
        if (!mask) continue;
        uint32_t any = 0;
        for (int w = tid; w < a.W && !any; w += kRuleThreads) {
            any = __ldg(mask + w);
            if (w == a.W - 1 && (a.V & 31)) any &= (1u << (a.V & 31)) - 1u;
        }
        if (!__syncthreads_or(any != 0) && tid == 0) bits |= SV_ROW_EMPTY_MASK;
    }
    if (bits) atomicOr(a.status, bits);
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
    sv::RuleArgs a = {};
    if (const sv_history *h = rules->history) {
        if (!h->prompt_bits || !h->output_bits || !h->output_counts) return SV_ERR_ARG;
        if (h->R < 1 || h->V != V || (!rules->slots && B > h->R)) return SV_ERR_SHAPE;
        a.prompt = h->prompt_bits;
        a.output = h->output_bits;
        a.counts = h->output_counts;
        a.R = h->R;
    }
    if (rules->bias_begin && (rules->n_bias < 0 ||
                              (rules->n_bias > 0 && (!rules->bias_tokens || !rules->bias_values))))
        return SV_ERR_ARG;
    if (rules->mask) {
        if (rules->n_masks < 1) return SV_ERR_ARG;
        if (!rules->mask_index && static_cast<long long>(B) * P > rules->n_masks) return SV_ERR_SHAPE;
    }
    a.in = static_cast<const char *>(logits);
    a.out = static_cast<char *>(out);
    a.B = B; a.P = P; a.V = V; a.v0 = v0; a.Vs = Vs;
    a.W = (V + 31) / 32;
    a.nchunk = (Vs + sv::kChunk - 1) / sv::kChunk;
    a.drafts = K > 0 ? draft_tokens : nullptr;
    a.K = K; a.pos0 = pos0;
    a.lengths = lengths; a.extra = extra;
    a.slots = rules->slots;
    a.rep = rules->repetition; a.freq = rules->frequency; a.pres = rules->presence;
    a.bias_begin = rules->n_bias > 0 ? rules->bias_begin : nullptr;
    a.bias_tokens = rules->bias_tokens; a.bias_values = rules->bias_values;
    a.n_bias = rules->n_bias;
    a.mask = rules->mask; a.n_masks = rules->n_masks; a.mask_index = rules->mask_index;
    a.status = status;
    const long long grid = static_cast<long long>(B) * a.nchunk;
    if (grid > INT_MAX) return SV_ERR_SHAPE;
    const bool in_place = in_at == out_at;
    auto *kernel = dtype == SV_F32 ? (in_place ? sv::rules_kernel<4, true> : sv::rules_kernel<4, false>)
                                   : (in_place ? sv::rules_kernel<2, true> : sv::rules_kernel<2, false>);
    return sv::note_cuda(sv::launch_pdl(kernel, dim3(static_cast<unsigned>(grid)),
                                        dim3(sv::kRuleThreads), 0,
                                        static_cast<cudaStream_t>(stream), a));
}
