// sv_history.cu -- token history of the requests in flight: which tokens the
// prompt held, which were emitted and how often.  The state behind the
// penalties of sv_logits_process, advanced by the tokens sv_verify emits.
//
// A slot is two bit planes over the vocabulary (prompt, output) and one count
// per token.  The planes are what a reader scans (V / 8 bytes instead of 4 V
// bytes of counts); a count is looked up only where its bit is set.
//
// At serving sizes history_add is bound by its launch: 64 prompts of up to 4096
// tokens take 6.6 us cold under a profiler, and calls from Python take 5 us back to
// back, what issuing them costs.  A reset reads V / 8 bytes of output bits a slot,
// writes twice that, and zeroes the counts of the tokens that were emitted, each in
// a sector of its own.  With L2 flushed, V = 129280: 4 slots 6 us, 256 slots 11
// (after 800 emitted tokens each; 17 after 4000), 2048 slots 55.
#include <climits>
#include <cstdint>

#include "sv.h"
#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

struct HistoryArgs {
    uint32_t *prompt, *output;
    int32_t *counts;
    int R, V, W;
    const int32_t *slots;
    const int32_t *tokens, *lens;
    int S, extra;
    long long n;             // B * S entries, or slots to reset
    int32_t *status;
};

__device__ __forceinline__ void raise_bits(int32_t *status, int bits) {
    if (status && bits) atomicOr(status, bits);
}

// One thread per (row, token) entry.  The prompt bit is tested before it is
// set: most prompt tokens repeat, and a plain load is cheaper than an atomic
// (a stale 0 only costs the atomic).
__global__ void __launch_bounds__(256) history_add_kernel(HistoryArgs a, int kind) {
    griddep_wait();
    griddep_launch_dependents();
    for (long long q = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; q < a.n;
         q += static_cast<long long>(gridDim.x) * blockDim.x) {
        const int b = static_cast<int>(q / a.S), s = static_cast<int>(q - static_cast<long long>(b) * a.S);
        const long long len = a.lens ? static_cast<long long>(__ldg(a.lens + b)) + a.extra : a.S;
        if (len < 0 || len > a.S) {
            if (s == 0) raise_bits(a.status, SV_ROW_BAD_LENGTH);
            continue;
        }
        if (s >= len) continue;
        const int slot = a.slots ? __ldg(a.slots + b) : b;
        if (slot < 0 || slot >= a.R) {
            if (s == 0) raise_bits(a.status, SV_ROW_BAD_SLOT);
            continue;
        }
        const int v = __ldg(a.tokens + q);
        if (v < 0 || v >= a.V) {
            raise_bits(a.status, SV_ROW_BAD_TOKEN);
            continue;
        }
        const uint32_t bit = 1u << (v & 31);
        uint32_t *word = (kind == SV_HISTORY_PROMPT ? a.prompt : a.output) +
                         static_cast<long long>(slot) * a.W + (v >> 5);
        if (kind == SV_HISTORY_PROMPT) {
            if (!(__ldcg(word) & bit)) atomicOr(word, bit);
        } else {
            atomicOr(word, bit);
            atomicAdd(a.counts + static_cast<long long>(slot) * a.V + v, 1);
        }
    }
}

// One thread per (slot, word).
__global__ void __launch_bounds__(256) history_reset_kernel(HistoryArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const long long total = a.n * a.W;
    for (long long q = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; q < total;
         q += static_cast<long long>(gridDim.x) * blockDim.x) {
        const long long r = q / a.W;
        const int w = static_cast<int>(q - r * a.W);
        const int slot = a.slots ? __ldg(a.slots + r) : static_cast<int>(r);
        if (slot < 0 || slot >= a.R) {
            if (w == 0) raise_bits(a.status, SV_ROW_BAD_SLOT);
            continue;
        }
        const long long at = static_cast<long long>(slot) * a.W + w;
        int32_t *counts = a.counts + static_cast<long long>(slot) * a.V + 32ll * w;
        // A slot listed twice: whichever thread sees the bits clears the counts.
        for (uint32_t m = a.output[at]; m; m &= m - 1) {
            const int i = __ffs(m) - 1;
            if (32ll * w + i < a.V) counts[i] = 0;
        }
        a.output[at] = 0;
        a.prompt[at] = 0;
    }
}

static sv_status history_check(const sv_history *h) {
    if (!h || !h->prompt_bits || !h->output_bits || !h->output_counts) return SV_ERR_ARG;
    if (misaligned4(h->prompt_bits, h->output_bits, h->output_counts)) return SV_ERR_ARG;
    if (h->R < 1 || h->V < 1 || h->V > SV_MAX_V) return SV_ERR_SHAPE;
    return SV_OK;
}

static HistoryArgs history_args(const sv_history *h) {
    HistoryArgs a = {};
    a.prompt = h->prompt_bits;
    a.output = h->output_bits;
    a.counts = h->output_counts;
    a.R = h->R;
    a.V = h->V;
    a.W = (h->V + 31) / 32;
    return a;
}

static int grid_of(long long threads, int block) {
    const long long g = (threads + block - 1) / block;
    return static_cast<int>(g < 148 * 64 ? g : 148 * 64);
}

}  // namespace sv

extern "C" sv_status sv_history_add(const sv_history *history, const int32_t *slots, int B,
                                    const int32_t *tokens, int S, const int32_t *lens, int extra,
                                    sv_history_kind kind, int32_t *status, void *stream) {
    sv::NvtxRange nvtx_range("sv_history_add");
    if (const sv_status e = sv::history_check(history)) return e;
    if (kind != SV_HISTORY_PROMPT && kind != SV_HISTORY_OUTPUT) return SV_ERR_ARG;
    if (B < 0 || S < 0 || (!slots && B > history->R)) return SV_ERR_SHAPE;
    if (B == 0 || S == 0) return SV_OK;
    if (!tokens || sv::misaligned4(slots, tokens, lens, status)) return SV_ERR_ARG;
    sv::HistoryArgs a = sv::history_args(history);
    a.slots = slots;
    a.tokens = tokens;
    a.lens = lens;
    a.S = S;
    a.extra = extra;
    a.n = static_cast<long long>(B) * S;
    a.status = status;
    return sv::note_cuda(sv::launch_pdl(sv::history_add_kernel, dim3(sv::grid_of(a.n, 256)), dim3(256),
                                        0, static_cast<cudaStream_t>(stream), a,
                                        static_cast<int>(kind)));
}

extern "C" sv_status sv_history_reset(const sv_history *history, const int32_t *slots, int n,
                                      int32_t *status, void *stream) {
    sv::NvtxRange nvtx_range("sv_history_reset");
    if (const sv_status e = sv::history_check(history)) return e;
    if (n < 0 || (!slots && n > history->R)) return SV_ERR_SHAPE;
    if (n == 0) return SV_OK;
    if (sv::misaligned4(slots, status)) return SV_ERR_ARG;
    sv::HistoryArgs a = sv::history_args(history);
    a.slots = slots;
    a.n = n;
    a.status = status;
    return sv::note_cuda(sv::launch_pdl(sv::history_reset_kernel, dim3(sv::grid_of(a.n * a.W, 256)),
                                        dim3(256), 0, static_cast<cudaStream_t>(stream), a));
}
