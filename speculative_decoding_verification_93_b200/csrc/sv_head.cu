// sv_head.cu -- output head with 4-bit weights and group scales on the
// tensor cores (tcgen05; the formula stands at sv_head_w4 in include/sv.h).
//
// The product is computed transposed: D[v, token] = sum_k W[v, k] x[token, k]
// with 128 vocabulary rows as the matrix unit's M and the tokens as its N,
// so that few tokens waste little and every weight is read once for up to 192 tokens.
//
// Exactness.  code - zero is an integer of at most five bits, exact in bf16,
// and so is its product with a bf16 x in fp32.  The scale is not folded into
// the bf16 operand (that would round every weight to 8 bits); instead each
// group's sum is read back from tensor memory, multiplied by its scale in
// fp32 and added to fp32 accumulators in registers.
//
// Up to 16 tokens take few_kernel (section 4), one launch.  Otherwise one launch
// packs the scheduled tokens of x into the operand layout (pack_kernel); the
// second (head_kernel) is persistent, one CTA per SM, and walks 128-row tiles of
// the vocabulary, K in stages of AK (256, or 128 above 64 tokens):
//   warp 0      asks for each stage's codes (one TMA tile, swizzled);
//   warp 2      copies each stage's x image (bulk copies);
//   warp 3      fetches scales and zero points into a ring of their own;
//   warp 1      issues tcgen05.mma, A from tensor memory, B from shared
//               memory, one batch per group and half of the tokens;
//   one or two warpgroups own one weight row per thread: they widen codes to
//               bf16 integers and write them to tensor memory as A;
//   two warpgroups read each finished batch back, scale and accumulate it, and
//               write the logits: up to 128 tokens by turns (every second
//               group each, the sums added at the end), above that one for
//               each half of the tokens.
// A vocabulary of few tiles has every tile's k shared out over several CTAs, whose
// sums join_kernel adds in their order.
// A in tensor memory keeps the widened weights (four times the bytes of the
// codes) out of shared memory, whose bandwidth the B operand needs.
//
// Measured, V x H = 129280 x 4096, bf16 out, groups of 128 / 64 / 32 (the last
// two with zero points), 600 calls over three heads in turn (on another board the
// forms above 64 tokens took up to a tenth more, under its power cap):
//      1 token   57 /  83 / 135 us (273 MB for groups of 128: 4.8 TB/s)
//      9 tokens  80 / 111 / 154
//     32 tokens  89 / 122 / 175
//     64 tokens 103 / 134 / 206
//    128 tokens 160 / 204 / 275
//    192 tokens 208 / 247 / 381 (203 GFLOP: 0.98 PFLOP/s for groups of 128)
//    200 tokens 335 / 420 / 676 (a second pass)
// Every group costs a round of hand-overs (products, read-back, buffer free),
// some 250 cycles whatever its length, and every 128 k a widening warpgroup
// some 1000: neither memory nor the matrix unit (16 cycles a product at 32
// tokens, 50 at 96, measured by issuing each twice) sets the pace before 192
// tokens, where the unit is half busy.
#include <atomic>
#include <climits>
#include <cstdint>
#include <cuda.h>

#include "sv.h"
#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

// ---------------------------------------------------------------------------
// Layout shared by both kernels.
// ---------------------------------------------------------------------------
constexpr int kTileV = 128;              // vocabulary rows per tile

// Tokens are taken in `passes` of `per` tokens, each pass in one or two
// `halves` of `nh` (a multiple of 16) tokens.  The x image of (pass, stage) holds, per half,
// blocks of nh rows x 64 k in the 128-byte swizzle.
struct TokenPlan {
    int count, passes, per, nh;
};

__host__ __device__ __forceinline__ TokenPlan token_plan(int count, int halves, int nh_max) {
    TokenPlan p;
    p.count = count;
    const int most = halves * nh_max, unit = 16 * halves;
    p.passes = (count + most - 1) / most;
    const int share = p.passes ? (count + p.passes - 1) / p.passes : 1;
    p.per = (share + unit - 1) / unit * unit;
    p.nh = p.per / halves;
    return p;
}

struct HeadArgs {
    const uint8_t *codes;
    const void *scale;
    const uint8_t *zero;
    bool scale_f32, out_f32;
    int V, H, group, G, tiles;
    int ak, nkb;         // k per stage, stages of a row
    const __nv_bfloat16 *x;
    int B, P;
    const int32_t *lengths;
    int extra;
    void *out;
    int halves, nh_max;
    int *count;          // workspace: scheduled tokens
    int *rows;           // workspace [B * P]: output row of each packed token
    char *image;         // workspace: x images
    int splits;          // of a row's k, each a CTA's; above 1 their sums are joined by join_kernel
    float *part;         // workspace [splits, B * P, tiles, 128]: sums of each
    int32_t *status;
};

// ---------------------------------------------------------------------------
// 1. Pack: the scheduled tokens, in order, in the operand layout.
// ---------------------------------------------------------------------------
constexpr int kPackThreads = 256;
constexpr int kPackGrid = 296;           // at most; two CTAs per SM
constexpr int kPackList = (1 << 20) / kPackGrid + 2;

__device__ __forceinline__ int row_positions(const HeadArgs &a, int b) {
    if (!a.lengths) return a.P;
    const long long n = static_cast<long long>(__ldg(a.lengths + b)) + a.extra;
    return static_cast<int>(max(0ll, min(n, static_cast<long long>(a.P))));
}

// Every CTA scans the lengths (a token's place is the sum of the lengths
// before it) and packs the tokens whose place is its index modulo the grid.
__global__ void __launch_bounds__(kPackThreads) pack_kernel(HeadArgs a) {
    __shared__ int place[kPackList], src[kPackList];
    __shared__ int wsum[kPackThreads / 32];
    __shared__ int mine;
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) mine = 0;
    __syncthreads();
    int run = 0;
    const int grid = gridDim.x;
    for (int b0 = 0; b0 < a.B; b0 += kPackThreads) {
        const int b = b0 + tid;
        const int n = b < a.B ? row_positions(a, b) : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int before = run, all = 0;
#pragma unroll
        for (int w = 0; w < kPackThreads / 32; ++w) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
        const int first = before + incl - n;
        // the first place >= first that this CTA packs
        int p = static_cast<int>(blockIdx.x) - first % grid;
        if (p < 0) p += grid;
        for (; p < n; p += grid) {
            const int at = atomicAdd(&mine, 1);
            place[at] = first + p;
            src[at] = b * a.P + p;
        }
        run += all;
        __syncthreads();
    }
    const TokenPlan t = token_plan(run, a.halves, a.nh_max);
    if (blockIdx.x == 0 && tid == 0) *a.count = run;
    const int chunks = a.H / 8;          // 16-byte chunks of one token
    const int total = mine * chunks;
    for (int q = tid; q < total; q += kPackThreads) {
        const int i = q / chunks, c = q - i * chunks;
        const int slot = place[i], pass = slot / t.per, in = slot - pass * t.per;
        const int half = in / t.nh, r = in - half * t.nh;
        if (c == 0) a.rows[slot] = src[i];
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(a.x + static_cast<long long>(src[i]) * a.H) + c);
        // k order 0 4 1 5 2 6 3 7: the order in which one shift of a code
        // word gives two codes (bits 0-3 and 16-19).
        uint4 w;
        w.x = __byte_perm(u.x, u.z, 0x5410);
        w.y = __byte_perm(u.x, u.z, 0x7632);
        w.z = __byte_perm(u.y, u.w, 0x5410);
        w.w = __byte_perm(u.y, u.w, 0x7632);
        const int per_stage = a.ak / 8, kb = c / per_stage, sub = (c % per_stage) / 8, col = c & 7;
        char *d = a.image + (static_cast<long long>(pass) * a.nkb + kb) * t.per * a.ak * 2 +
                  (half * (a.ak / 64) + sub) * t.nh * 128 + r * 128 + ((col ^ (r & 7)) * 16);
        *reinterpret_cast<uint4 *>(d) = w;
    }
}

// ---------------------------------------------------------------------------
// 2. Tensor-core primitives (PTX ISA, tcgen05).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t *smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem)),
                 "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups
// 1024 bytes apart; the low word holds the address.
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr) { return ((addr & 0x3ffffu) >> 4) | (1u << 16); }

// The matrix unit's instructions are issued by one lane, elected inside the
// statement: the warp itself never diverges, so the operands stay in uniform
// registers and nothing has to reconverge.
// D (fp32, tensor memory) (+)= A (bf16, tensor memory) * B (bf16, shared
// memory), over 32 or 64 k of one swizzled block: products of 16.
template <int K>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool add) {
    if constexpr (K == 64)
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b0, b1, b2, b3;\n\t.reg .b32 l1, l2, l3, c1, c2, c3;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 t, %4, %4;\n\t"
            "add.u32 l1, %2, 2;\n\tadd.u32 l2, %2, 4;\n\tadd.u32 l3, %2, 6;\n\t"
            "add.u32 c1, %1, 8;\n\tadd.u32 c2, %1, 16;\n\tadd.u32 c3, %1, 24;\n\t"
            "mov.b64 b0, {%2, %3};\n\tmov.b64 b1, {l1, %3};\n\tmov.b64 b2, {l2, %3};\n\tmov.b64 b3, {l3, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %4, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c1], b1, %4, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c2], b2, %4, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c3], b3, %4, t;\n\t}"
            ::"r"(d), "r"(a), "r"(b_lo), "n"(kDescHigh), "r"(idesc), "r"(static_cast<uint32_t>(add)) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b0, b1;\n\t.reg .b32 l1, c1;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 t, %4, %4;\n\t"
            "add.u32 l1, %2, 2;\n\tadd.u32 c1, %1, 8;\n\tmov.b64 b0, {%2, %3};\n\tmov.b64 b1, {l1, %3};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %4, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c1], b1, %4, t;\n\t}"
            ::"r"(d), "r"(a), "r"(b_lo), "n"(kDescHigh), "r"(idesc), "r"(static_cast<uint32_t>(add)) : "memory");
}
// `bar` completes one arrival when every product issued so far has finished.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&f)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]),
          "=f"(f[8]), "=f"(f[9]), "=f"(f[10]), "=f"(f[11]), "=f"(f[12]), "=f"(f[13]), "=f"(f[14]), "=f"(f[15]),
          "=f"(f[16]), "=f"(f[17]), "=f"(f[18]), "=f"(f[19]), "=f"(f[20]), "=f"(f[21]), "=f"(f[22]), "=f"(f[23]),
          "=f"(f[24]), "=f"(f[25]), "=f"(f[26]), "=f"(f[27]), "=f"(f[28]), "=f"(f[29]), "=f"(f[30]), "=f"(f[31])
        : "r"(addr) : "memory");
}
// Loads from tensor memory land by the wait; naming their registers here
// keeps every use behind it.
__device__ __forceinline__ void tc_wait_ld(float (&f)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3]), "+f"(f[4]), "+f"(f[5]), "+f"(f[6]), "+f"(f[7]),
                   "+f"(f[8]), "+f"(f[9]), "+f"(f[10]), "+f"(f[11]), "+f"(f[12]), "+f"(f[13]), "+f"(f[14]), "+f"(f[15]),
                   "+f"(f[16]), "+f"(f[17]), "+f"(f[18]), "+f"(f[19]), "+f"(f[20]), "+f"(f[21]), "+f"(f[22]), "+f"(f[23]),
                   "+f"(f[24]), "+f"(f[25]), "+f"(f[26]), "+f"(f[27]), "+f"(f[28]), "+f"(f[29]), "+f"(f[30])
                 :: "memory");
    asm volatile("" : "+f"(f[31]));
}
template <int N> __device__ __forceinline__ void regs_less() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// One tile of a two-dimensional tensor map into shared memory.
__device__ __forceinline__ void tma_tile(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}

// ---------------------------------------------------------------------------
// 3. The product.
// ---------------------------------------------------------------------------
constexpr uint32_t kTmemCols = 512;
constexpr int kParGroups = 8;            // groups per chunk of the parameter ring
constexpr int kParSlots = 3;
constexpr int kDone = 8;                 // ring of stage-done barriers
constexpr uint64_t kHeadWaitNs = 1000000000ull;

// Scale and zero point of kParGroups groups of a tile's rows.  `off` is the
// pair -zero / 64 in bf16 (see widen8).
struct ParChunk {
    float scale[kParGroups][kTileV];
    uint32_t off[kParGroups][kTileV];
};

// HALVES of up to NH tokens, for weights in groups of GROUP.  AK k per stage, AS
// A operands in tensor memory (AK / 2 columns each, behind the accumulators),
// CS and XS stages of codes and x in shared memory, WW warpgroups that widen.
// A batch is one group of one half.  Two halves: an accumulating warpgroup and
// two batches in tensor memory for each.  One half: the two warpgroups take its
// batches by turns, four (NH = 128: three) in tensor memory.
//   NH <= 64: stages of 256 k, which two warpgroups widen in turn.
//   NH > 64: the accumulators need the registers of a second widening
//   warpgroup, and 384 columns of batches leave A two stages of 128 k.
// One half is the faster form wherever its batches fit (three at least): two
// halves of 64 took 150 / 213 / 366 us at 128 tokens, two of 16 135 / 217 / 357
// at 17.
template <int HALVES, int NH, int GROUP> struct HeadCfg {
    static constexpr int kHalves = HALVES, kNh = NH;
    static constexpr int AK = NH <= 64 ? 256 : 128;
    static constexpr int AS = 2;
    static constexpr int WW = NH <= 64 ? 2 : 1;
    static constexpr int DB = NH == 128 ? 3 : 4 / HALVES;   // batches of a half in tensor memory
    static constexpr int XS = 2;
    static constexpr int CS = NH <= 64 ? 4 : 8;
    static constexpr int kSubs = AK / GROUP;
    static constexpr int kACol = HALVES * DB * NH;
    static constexpr int kThreads = 128 * (3 + WW);
    // Registers a thread of the service, widening and accumulating
    // warpgroups: their sum stays within what the CTA was launched with.
    static constexpr int kRegs0 = 72;
    static constexpr int kRegsW = NH <= 64 ? 80 : 72;
    static constexpr int kRegsA = NH <= 64 ? 120 : 184;
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static_assert(kRegs0 + WW * kRegsW + 2 * kRegsA <= (3 + WW) * kLaunchRegs, "register split");
    static constexpr int kCodeBytes = kTileV * AK / 2;
    static constexpr int kXBytes = HALVES * NH * AK * 2;
    // One half: what the accumulating warpgroups hand each other.
    static constexpr int kSums = HALVES == 1 ? NH / 2 * kTileV : 0;
    // More than half of the SM's shared memory, as two CTAs on one SM would
    // wait for each other's tensor memory.
    static constexpr int kUsed = 1024 + XS * kXBytes + CS * kCodeBytes +
                                 kParSlots * static_cast<int>(sizeof(ParChunk)) + 2 * kSums * 4;
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static_assert(kSmem <= 227 * 1024 - 1024, "shared memory");
    static_assert(kACol + AS * AK / 2 <= static_cast<int>(kTmemCols), "tensor memory");
    static_assert(XS < kDone && AS < kDone && AS % WW == 0, "rings");
};

struct HeadBars {
    uint64_t cfull[8], cempty[8];        // codes landed; read by the widening warps
    uint64_t xfull[2];                   // x landed
    uint64_t afull[2];                   // A written
    uint64_t done[kDone];                // the matrix unit is through a stage: its x and A are free
    uint64_t dfull[4], dempty[4];        // a batch finished; read back
    uint64_t pfull[kParSlots], pempty[kParSlots];
    uint64_t sums, summed;               // one half: both warpgroups' sums of a job are in shared memory; read
    uint32_t tmem;
};

// Bounded wait, warp-wide: every lane gets the same answer.  One compact loop:
// five roles share each scheduler's instruction cache, and a role's pace is
// set by how much of its code has to be fetched again.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    uint64_t t0 = 0;
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, now - t0 > kHeadWaitNs)) return false;
    }
    return true;
}

// A CTA's share of a row's k: stages k0 .. k0 + nkb - 1, groups g0 .. g0 + G - 1.
// Shares are whole chunks of kParGroups groups.
struct Span {
    int split, k0, nkb, g0, G;
};

__host__ __device__ __forceinline__ Span span_of(int split, int splits, int G, int nkb, int subs) {
    const int chunks = (G + kParGroups - 1) / kParGroups, per = kParGroups / subs;   // stages of a chunk
    const int c0 = chunks * split / splits, c1 = chunks * (split + 1) / splits;
    Span p;
    p.split = split;
    p.g0 = c0 * kParGroups;
    p.G = (c1 * kParGroups < G ? c1 * kParGroups : G) - p.g0;
    p.k0 = c0 * per;
    p.nkb = (c1 * per < nkb ? c1 * per : nkb) - p.k0;
    return p;
}

__device__ __forceinline__ int warp_value(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Eight codes to four pairs (code - zero) / 64 in bf16, exact.  A code in the
// low bits of a bf16 is the number code * 2^-133 (bits 0-3) or code * 2^-129
// (bits 4-7): below the normal numbers, where the format is linear, up to
// 2^-126 * 2.  So one mask takes out two codes, and one fused multiply-add by
// 2^127 (2^123) subtracts the zero point with no exponent to set first: five
// integer operations, which run at half the rate of the others, for eight
// codes, against seven when 128 is OR-ed in.  The factor 64 is in the scale.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t off, uint32_t *r) {
    const uint32_t h = w >> 8;
    const uint32_t p[4] = {w & 0x000f000fu, w & 0x00f000f0u, h & 0x000f000fu, h & 0x00f000f0u};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r[i]) : "r"(p[i]), "r"(i & 1 ? 0x7d007d00u : 0x7f007f00u), "r"(off));
}

__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
    const __nv_bfloat162 p = __float2bfloat162_rn(static_cast<float>(z) * (-1.f / 64.f));   // exact
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ float ld_scale(const HeadArgs &a, long long at) {
    return a.scale_f32 ? __ldg(static_cast<const float *>(a.scale) + at)
                       : ld_elem<2>(static_cast<const char *>(a.scale), at);
}

// Codes of every stage (one lane).  start() asks for the first tile's before
// the token count is known.
template <typename Cfg> struct CodeCopy {
    const Span &span;
    const CUtensorMap *map;
    HeadBars &bar;
    char *ring;
    int tile0, s = 0;
    __device__ CodeCopy(const Span &p, const CUtensorMap *m, HeadBars &b, char *r, int tile)
        : span(p), map(m), bar(b), ring(r), tile0(tile) {}
    __device__ __forceinline__ void copy(int tile, int kb) {
        const int slot = s % Cfg::CS;
        mbar_arrive_expect_tx(&bar.cfull[slot], Cfg::kCodeBytes);
        tma_tile(ring + slot * Cfg::kCodeBytes, map, (span.k0 + kb) * (Cfg::AK / 2), tile * kTileV, &bar.cfull[slot]);
        ++s;
    }
    __device__ void start() {
        for (int kb = 0; kb < min(span.nkb, Cfg::CS); ++kb) copy(tile0, kb);
    }
    __device__ bool run(const TokenPlan &t, int jobs) {
        bool ok = true;
        int q = 0;
        for (int job = 0; ok && job < jobs; ++job) {
            const int tile = tile0 + job / t.passes * gridDim.x;
            for (int kb = 0; kb < span.nkb; ++kb, ++q) {
                if (q < s) continue;      // asked for by start()
                if (!mbar_wait(&bar.cempty[s % Cfg::CS], ((s / Cfg::CS) & 1) ^ 1, kHeadWaitNs)) { ok = false; break; }
                copy(tile, kb);
            }
        }
        // The copies in flight land before this CTA may leave.
        for (int i = max(0, s - Cfg::CS); i < s; ++i)
            mbar_wait(&bar.cfull[i % Cfg::CS], (i / Cfg::CS) & 1, kHeadWaitNs);
        return ok;
    }
};

// The x images of every stage (one lane).
template <typename Cfg>
__device__ bool x_role(const HeadArgs &a, const Span &span, const TokenPlan &t, int jobs, HeadBars &bar, char *xring) {
    const uint32_t bytes = t.per * Cfg::AK * 2;
    bool ok = true;
    int s = 0;
    for (int job = 0; ok && job < jobs; ++job) {
        const char *src = a.image + (static_cast<long long>(job % t.passes) * a.nkb + span.k0) * bytes;
        for (int kb = 0; kb < span.nkb; ++kb, ++s) {
            const int slot = s % Cfg::XS, old = s - Cfg::XS;
            if (old >= 0 && !mbar_wait(&bar.done[old % kDone], (old / kDone) & 1, kHeadWaitNs)) { ok = false; break; }
            mbar_arrive_expect_tx(&bar.xfull[slot], bytes);
            bulk_g2s(xring + slot * Cfg::kXBytes, src + static_cast<long long>(kb) * bytes, bytes, &bar.xfull[slot]);
        }
    }
    for (int q = max(0, s - Cfg::XS); q < s; ++q)
        mbar_wait(&bar.xfull[q % Cfg::XS], (q / Cfg::XS) & 1, kHeadWaitNs);
    return ok;
}

// The matrix unit's instructions (warp 1, all lanes together).  Every
// stage has all its batches; one past the last group has no products.
template <typename Cfg, int GROUP>
__device__ bool mma_role(const HeadArgs &a, const Span &span, const TokenPlan &t, int jobs, HeadBars &bar, const char *xring,
                         uint32_t tmem) {
    const uint32_t nh = warp_value(t.nh), nh8 = nh * 8;
    constexpr int NH = Cfg::kNh;
    const int nkb = warp_value(span.nkb), stages = warp_value(jobs) * nkb;
    const int last_subs = warp_value(span.G) - (nkb - 1) * Cfg::kSubs;   // groups of the last stage
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((nh >> 3) << 17) | ((kTileV >> 4) << 24);
    const uint32_t x0 = smem_desc(smem_u32(xring));
    constexpr int kUnit = GROUP < 64 ? GROUP : 64;
    int left = nkb;                       // stages of the job still to come
    uint32_t i = 0;                       // batch of a half
    bool ok = true;
#pragma unroll 1
    for (uint32_t s = 0; ok && s < static_cast<uint32_t>(stages); ++s) {
        const uint32_t ab = s % Cfg::AS, slot = s % Cfg::XS;
        const int subs = left == 1 ? last_subs : Cfg::kSubs;
        const uint32_t xs = x0 + slot * (Cfg::kXBytes / 16);
        uint32_t acol = tmem + Cfg::kACol + ab * (Cfg::AK / 2);
        int k32 = 0;                      // 32-k blocks into the stage
        if (!warp_wait(&bar.xfull[slot], (s / Cfg::XS) & 1) || !warp_wait(&bar.afull[ab], (s / Cfg::AS) & 1)) {
            ok = false;
            break;
        }
#pragma unroll 1
        for (int j = 0; j < Cfg::kSubs; ++j, ++i) {
            const uint32_t d = i % Cfg::DB;
            const uint32_t parity = ((i / Cfg::DB) & 1) ^ 1;
            if (!warp_wait(&bar.dempty[d], parity) ||
                (Cfg::kHalves == 2 && !warp_wait(&bar.dempty[Cfg::DB + d], parity))) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < Cfg::kHalves; ++h) {
                const uint32_t acc = tmem + (h * Cfg::DB + d) * NH, xh = xs + h * (Cfg::AK / 64) * nh8;
                if (j < subs) {
#pragma unroll
                    for (int w = 0; w < GROUP / kUnit; ++w) {
                        const int k = k32 + w * kUnit / 32;   // 32-k block of the stage
                        mma_ts<kUnit>(acc, acol + 16 * (k - k32), xh + (k >> 1) * nh8 + (k & 1) * 4, idesc, w > 0);
                    }
                }
                mma_commit(&bar.dfull[h * Cfg::DB + d]);
            }
            acol += GROUP / 2;
            k32 += GROUP / 32;
        }
        if (!ok) break;
        mma_commit(&bar.done[s % kDone]);
        if (--left == 0) left = nkb;
    }
    // Nothing of the matrix unit is in flight when tensor memory is freed: the
    // last stage's commit covers all before it.  After a wait that ran out,
    // a millisecond is far more than what was issued needs.
    if (!ok)
        for (const uint64_t t0 = global_ns(); global_ns() - t0 < 1000000;) __nanosleep(1000);
    return ok && (stages == 0 || warp_wait(&bar.done[(stages - 1) % kDone], ((stages - 1) / kDone) & 1));
}

// Scales and zero points (warp 3, four rows a lane): as fp32 and bf16 pairs
// in shared memory, eight groups at a time, so that the rows' strided reads
// are 16 and 8 bytes wide where the alignment allows it, made once for both
// halves, and ahead of their use.
__device__ bool param_role(const HeadArgs &a, const Span &span, const TokenPlan &t, int jobs, int tile0, HeadBars &bar,
                           ParChunk *ring) {
    constexpr int kRows = kTileV / 32;
    const int lane = threadIdx.x & 31;
    const bool wide = !a.scale_f32 && a.G % 8 == 0 && (reinterpret_cast<uintptr_t>(a.scale) & 15) == 0 &&
                      (reinterpret_cast<uintptr_t>(a.zero) & 7) == 0;
    int c = 0;
    for (int job = 0; job < jobs; ++job) {
        const int tile = tile0 + job / t.passes * gridDim.x;
        for (int g0 = 0; g0 < span.G; g0 += kParGroups, ++c) {
            ParChunk &p = ring[c % kParSlots];
            long long at[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                at[r] = static_cast<long long>(min(tile * kTileV + r * 32 + lane, a.V - 1)) * a.G + span.g0 + g0;
            if (wide) {
                uint4 u[kRows];
                uint2 z[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    u[r] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.scale) + at[r]));
                    z[r] = a.zero ? __ldg(reinterpret_cast<const uint2 *>(a.zero + at[r])) : make_uint2(0, 0);
                }
                if (!warp_wait(&bar.pempty[c % kParSlots], ((c / kParSlots) & 1) ^ 1)) return false;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const uint32_t w[4] = {u[r].x, u[r].y, u[r].z, u[r].w};
#pragma unroll
                    for (int q = 0; q < kParGroups; ++q) {
                        p.scale[q][r * 32 + lane] = 64.f * (q & 1 ? bf16_hi(w[q / 2]) : bf16_lo(w[q / 2]));
                        if (a.zero)
                            p.off[q][r * 32 + lane] = zero_pair((q < 4 ? z[r].x : z[r].y) >> (8 * (q & 3)) & 15u);
                    }
                }
            } else {
                if (!warp_wait(&bar.pempty[c % kParSlots], ((c / kParSlots) & 1) ^ 1)) return false;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
#pragma unroll
                    for (int q = 0; q < kParGroups; ++q) {
                        const long long e = at[r] + min(q, span.G - 1 - g0);
                        p.scale[q][r * 32 + lane] =
                            64.f * ld_scale(a, e);
                        if (a.zero) p.off[q][r * 32 + lane] = zero_pair(__ldg(a.zero + e) & 15u);
                    }
                }
            }
            mbar_arrive(&bar.pfull[c % kParSlots]);
        }
    }
    return true;
}

// One of WW warpgroups: the stages s = wi mod WW, one weight row a thread, 32 k
// (a piece) at a time.  The next piece's codes are read from shared memory while
// this one's are widened.  Four pieces to a round of the loop (17 tokens of
// 129280 x 4096, group 128: 89 us; two 93, one 99).
template <typename Cfg, int GROUP>
__device__ bool widen_role(const HeadArgs &a, const Span &span, int jobs, HeadBars &bar, const char *ring,
                           const ParChunk *par, uint32_t tmem, int wi) {
    constexpr int kRowBytes = Cfg::AK / 2, kPieces = Cfg::AK / 32, kEach = GROUP / 32;   // pieces of a stage, a group
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int stages = jobs * span.nkb, chunks = (span.G + kParGroups - 1) / kParGroups;
    const int r = quarter * 32 + lane;
    // The copy's swizzle: 16-byte pieces of 128-byte (64-byte) rows.
    const int swz = kRowBytes == 128 ? r & 7 : (r >> 1) & 3;
    const uint32_t dst0 = tmem + Cfg::kACol + (static_cast<uint32_t>(quarter * 32) << 16);
    int kb = wi, c0 = 0, have = -1;       // stage of the job, chunks before the job, chunk at hand
    uint32_t off = zero_pair(8);
    // Hand back chunk `have`, wait for the next one.
    auto next_chunk = [&](bool wait) {
        if (have >= 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.pempty[have % kParSlots]);
            __syncwarp();
        }
        ++have;
        return !wait || warp_wait(&bar.pfull[have % kParSlots], (have / kParSlots) & 1);
    };
    // Zero point of piece q of the stage at kb.
    auto zero_of = [&](int q) {
        const int gi = min(kb * Cfg::kSubs + q / kEach, span.G - 1), c = c0 + gi / kParGroups;
        while (have < c)
            if (!next_chunk(true)) return false;
        off = par[c % kParSlots].off[gi % kParGroups][r];
        return true;
    };
    const char *row = ring + r * kRowBytes;
    uint4 u;
    auto first = [&](int s) {             // of stage s
        if (!warp_wait(&bar.cfull[s % Cfg::CS], (s / Cfg::CS) & 1)) return false;
        row = ring + s % Cfg::CS * Cfg::kCodeBytes + r * kRowBytes;
        u = *reinterpret_cast<const uint4 *>(row + swz * 16);
        while (kb >= span.nkb) { kb -= span.nkb; c0 += chunks; }
        return !a.zero || zero_of(0);
    };
    if (wi < stages && !first(wi)) return false;
#pragma unroll 1
    for (int s = wi; s < stages; s += Cfg::WW) {
        const int ab = s % Cfg::AS, old = s - Cfg::AS;
        const uint32_t dst = dst0 + ab * (Cfg::AK / 2);
        if (old >= 0 && !warp_wait(&bar.done[old % kDone], (old / kDone) & 1)) return false;
        tc_fence_after();
#pragma unroll 4
        for (int q = 0; q < kPieces; ++q) {
            const uint4 v = u;
            const uint32_t o = off;
            if (q + 1 < kPieces) {
                u = *reinterpret_cast<const uint4 *>(row + (((q + 1) ^ swz) * 16));
                if (a.zero && (q + 1) % kEach == 0 && !zero_of(q + 1)) return false;
            }
            uint32_t w[16];
            widen8(v.x, o, w);
            widen8(v.y, o, w + 4);
            widen8(v.z, o, w + 8);
            widen8(v.w, o, w + 12);
            tmem_st16(dst + q * 16, w);
        }
        // A is written, and the stage's codes were read into registers.
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bar.afull[ab]);
            mbar_arrive(&bar.cempty[s % Cfg::CS]);
        }
        __syncwarp();
        kb += Cfg::WW;
        if (s + Cfg::WW < stages && !first(s + Cfg::WW)) return false;
    }
    if (a.zero)
        for (const int all = jobs * chunks; have < all;)
            if (!next_chunk(have + 1 < all)) return false;
    return true;
}

__device__ __forceinline__ void store_logit(float *p, float z) { *p = z; }
__device__ __forceinline__ void store_logit(__nv_bfloat16 *p, float z) { *p = __float2bfloat16_rn(z); }

// Adds a batch's first nh columns at `src` in tensor memory, scaled, to acc;
// the next columns are on their way while these are added.
template <typename Cfg>
__device__ __forceinline__ void add_batch(float (&acc)[Cfg::kNh], uint32_t src, float sc, int nh) {
    constexpr int L = 32, N = Cfg::kNh / L, kAhead = Cfg::kHalves == 2 ? 2 : 1;
    const float2 ss = make_float2(sc, sc);
    float d[kAhead][L];
    tmem_ld(src, d[0]);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (L * k < nh) {
            if (kAhead == 1 && k > 0) tmem_ld(src + L * k, d[0]);
            tc_wait_ld(d[k % kAhead]);
            if (kAhead == 2 && k + 1 < N && L * (k + 1) < nh) tmem_ld(src + L * (k + 1), d[(k + 1) % kAhead]);
#pragma unroll
            for (int n = 0; n < L; n += 2) {
                float *y = acc + L * k + n;
                const float2 z = __ffma2_rn(make_float2(d[k % kAhead][n], d[k % kAhead][n + 1]), ss, make_float2(y[0], y[1]));
                y[0] = z.x;
                y[1] = z.y;
            }
        }
    }
}

// Writes N of a row's logits, four neighbouring tokens at a time: those of
// tokens first + (n / 4) * step + n % 4, of which `live` exist.  One vocabulary
// row per lane: a warp writes 32 consecutive logits of each token.
template <int N, int ROWS, typename T>
__device__ __forceinline__ void write_logits(T *out, int V, const float (&y)[N], const int (&rows)[ROWS], int first,
                                             int step, int live, bool inside) {
#pragma unroll
    for (int n0 = 0; n0 < N; n0 += 4) {
        const int at = first + n0 / 4 * step;
        if (at < live) {
            T *to[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
                to[n] = out + static_cast<long long>(__shfl_sync(0xffffffffu, rows[n0 / 4 * step / 32], (at + n) % 32)) * V;
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (at + n < live && inside) store_logit(to[n], y[n0 + n]);
        }
    }
}

// The same for a share's sums, `next` apart from token to token.
template <int N>
__device__ __forceinline__ void write_share(float *to, long long next, const float (&y)[N], int first, int step, int live) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int at = first + n / 4 * step + n % 4;
        if (at < live) to[at * next] = y[n];
    }
}

// A thread owns one vocabulary row: of half h, or with one half of every second
// group (h, h + 2, ...).
template <typename Cfg>
__device__ bool accumulate_role(const HeadArgs &a, const Span &span, const TokenPlan &t, int jobs, int tile0, HeadBars &bar,
                                const ParChunk *par, float *sums, uint32_t tmem, int h) {
    constexpr int NH = Cfg::kNh, kRows = (NH + 31) / 32;
    constexpr bool kWhole = Cfg::kHalves == 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int batches = span.nkb * Cfg::kSubs;   // of a job and half; one past the last group has no products
    int i = 0, slot = 0, phase = 0;       // batch; slot and phase of the parameter ring
    for (int job = 0; job < jobs; ++job) {
        const int tile = tile0 + job / t.passes * gridDim.x, pass = job % t.passes;
        const int v = tile * kTileV + quarter * 32 + lane;
        // Output rows of these tokens, 32 to a register across the lanes.
        const int t0 = pass * t.per + (kWhole ? 0 : h * t.nh), live = min(t.nh, t.count - t0);
        int rows[kRows];
#pragma unroll
        for (int n = 0; n < kRows; ++n)
            rows[n] = 32 * n < live ? __ldg(a.rows + t0 + min(32 * n + lane, live - 1)) : 0;
        float acc[NH];
#pragma unroll
        for (int n = 0; n < NH; ++n) acc[n] = 0.f;
        constexpr int kStep = kWhole ? 2 : 1;
#pragma unroll 1
        for (int g0 = 0; g0 < span.G; g0 += kParGroups) {
            // This chunk's scales of the row; those past the last group are not used.
            if (!warp_wait(&bar.pfull[slot], phase)) return false;
            const float *scale = &par[slot].scale[kWhole ? h : 0][quarter * 32 + lane];
            const int n_batch = min(kParGroups, batches - g0);
#pragma unroll 1
            for (int j = kWhole ? h : 0; j < n_batch; j += kStep, scale += kStep * kTileV) {
                const int at = i + j, db = kWhole ? at % Cfg::DB : h * Cfg::DB + at % Cfg::DB;
                const float sc = *scale;
                if (!warp_wait(&bar.dfull[db], (at / Cfg::DB) & 1)) return false;
                tc_fence_after();
                if (g0 + j < span.G) add_batch<Cfg>(acc, lanes + db * NH, sc, t.nh);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.dempty[db]);
            }
            i += n_batch;
            if (lane == 0) mbar_arrive(&bar.pempty[slot]);
            if (++slot == kParSlots) { slot = 0; phase ^= 1; }
        }
        const bool inside = v < a.V;
        const long long vo = v;
        // A share's sums: token t0 + n of this tile.
        float *share = nullptr;
        if (a.splits > 1)
            share = a.part + ((static_cast<long long>(span.split) * a.B * a.P + t0) * a.tiles + tile) * kTileV + quarter * 32 + lane;
        const long long next = static_cast<long long>(a.tiles) * kTileV;
        if constexpr (kWhole) {
            // Each warpgroup takes every second four tokens of both.  (No
            // branches: code that runs once a job is fetched as it runs, and
            // straight lines are fetched ahead.)
            float *buf = sums + quarter * 32 + lane;
            if (job > 0 && !warp_wait(&bar.summed, (job - 1) & 1)) return false;
            float mine[NH / 2];
#pragma unroll
            for (int n = 0; n < NH / 2; ++n) {
                const int c = n / 4 * 8 + n % 4;
                buf[(1 - h) * Cfg::kSums + n * kTileV] = h ? acc[c] : acc[c + 4];
                mine[n] = h ? acc[c + 4] : acc[c];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.sums);
            if (!warp_wait(&bar.sums, job & 1)) return false;
#pragma unroll
            for (int n = 0; n < NH / 2; ++n) mine[n] += buf[h * Cfg::kSums + n * kTileV];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.summed);
            if (share) write_share(share, next, mine, 4 * h, 8, live);
            else if (a.out_f32) write_logits(static_cast<float *>(a.out) + vo, a.V, mine, rows, 4 * h, 8, live, inside);
            else write_logits(static_cast<__nv_bfloat16 *>(a.out) + vo, a.V, mine, rows, 4 * h, 8, live, inside);
        } else {
            if (share) write_share(share, next, acc, 0, 4, live);
            else if (a.out_f32) write_logits(static_cast<float *>(a.out) + vo, a.V, acc, rows, 0, 4, live, inside);
            else write_logits(static_cast<__nv_bfloat16 *>(a.out) + vo, a.V, acc, rows, 0, 4, live, inside);
        }
    }
    return true;
}

template <int HALVES, int NH, int GROUP>
__global__ void __launch_bounds__(HeadCfg<HALVES, NH, GROUP>::kThreads, 1)
head_kernel(HeadArgs a, const __grid_constant__ CUtensorMap map) {
    using Cfg = HeadCfg<HALVES, NH, GROUP>;
    extern __shared__ char dyn[];
    __shared__ HeadBars bar;
    char *xring = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    char *cring = xring + Cfg::XS * Cfg::kXBytes;
    ParChunk *par = reinterpret_cast<ParChunk *>(cring + Cfg::CS * Cfg::kCodeBytes);
    float *sums = reinterpret_cast<float *>(par + kParSlots);
    const int tid = threadIdx.x, warp = warp_value(tid >> 5), lane = tid & 31, wg = warp >> 2;
    // Whole rows, tile by tile, or (few tiles) one share of one tile.
    const int split = a.splits > 1 ? static_cast<int>(blockIdx.x) / a.tiles : 0;
    const int tile0 = static_cast<int>(blockIdx.x) - split * a.tiles;
    const Span span = span_of(split, a.splits, a.G, a.nkb, Cfg::kSubs);
    CodeCopy<Cfg> codes(span, &map, bar, cring, tile0);
    if (tid == 0) {
        for (int i = 0; i < Cfg::CS; ++i) { mbar_init(&bar.cfull[i], 1); mbar_init(&bar.cempty[i], 4); }
        for (int i = 0; i < Cfg::XS; ++i) mbar_init(&bar.xfull[i], 1);
        for (int i = 0; i < Cfg::AS; ++i) mbar_init(&bar.afull[i], 4);
        for (int i = 0; i < kDone; ++i) mbar_init(&bar.done[i], 1);
        for (int i = 0; i < 4; ++i) { mbar_init(&bar.dfull[i], 1); mbar_init(&bar.dempty[i], 4); }
        for (int i = 0; i < kParSlots; ++i) {
            mbar_init(&bar.pfull[i], 32);
            mbar_init(&bar.pempty[i], 8 + (a.zero ? 4 * Cfg::WW : 0));
        }
        mbar_init(&bar.sums, 8);
        mbar_init(&bar.summed, 8);
        fence_mbar_init();
        // The codes of the first stages are asked for at once: the pack
        // kernel let this grid launch after its own wait, so whatever ran
        // before this call has finished.
        codes.start();
    }
    if (warp == 1) tmem_alloc(&bar.tmem, kTmemCols);
    griddep_wait();
    griddep_launch_dependents();
    const TokenPlan t = token_plan(__ldcg(a.count), HALVES, NH);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = warp_value(bar.tmem);
    const int my_tiles = (a.tiles - tile0 + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    const int jobs = my_tiles * t.passes;
    bool ok = true;
    if (wg == 0) {
        regs_less<Cfg::kRegs0>();
        if (warp == 0) {
            if (lane == 0) ok = codes.run(t, jobs);
        } else if (warp == 1) {
            ok = mma_role<Cfg, GROUP>(a, span, t, jobs, bar, xring, tmem);
        } else if (warp == 2) {
            if (lane == 0) ok = x_role<Cfg>(a, span, t, jobs, bar, xring);
        } else {
            ok = param_role(a, span, t, jobs, tile0, bar, par);
        }
    } else if (wg <= Cfg::WW) {
        regs_less<Cfg::kRegsW>();
        ok = widen_role<Cfg, GROUP>(a, span, jobs, bar, cring, par, tmem, wg - 1);
    } else {
        regs_more<Cfg::kRegsA>();
        ok = accumulate_role<Cfg>(a, span, t, jobs, tile0, bar, par, sums, tmem, wg - 1 - Cfg::WW);
    }
    if (!ok && a.status) atomicOr(a.status, SV_NOTE_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free(tmem, kTmemCols);
}

// The shares' sums of each logit, in their order.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(HeadArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int slot = blockIdx.x, v = (blockIdx.y * kJoinThreads + threadIdx.x) * 4, width = a.tiles * kTileV;
    if (slot >= __ldcg(a.count) || v >= a.V) return;
    const long long next = static_cast<long long>(a.B) * a.P * width;
    const float *from = a.part + static_cast<long long>(slot) * width + v;
    float4 y = *reinterpret_cast<const float4 *>(from);
    for (int i = 1; i < a.splits; ++i) {
        const float4 z = *reinterpret_cast<const float4 *>(from + i * next);
        y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
    }
    const float w[4] = {y.x, y.y, y.z, y.w};
    const long long o = static_cast<long long>(__ldcg(a.rows + slot)) * a.V + v;
#pragma unroll
    for (int n = 0; n < 4; ++n)
        if (v + n < a.V) {
            if (a.out_f32) store_logit(static_cast<float *>(a.out) + o + n, w[n]);
            else store_logit(static_cast<__nv_bfloat16 *>(a.out) + o + n, w[n]);
        }
}

// ---------------------------------------------------------------------------
// 4. Few tokens: one launch, no tensor memory.
//
// With at most 16 tokens the hand-overs between roles above would set the pace
// (17 tokens of 129280 x 4096 take 89 us there).  Here a warp does all of it for
// 32 vocabulary rows, and what it costs is to widen them (one token, groups of 128:
// issue slots 59%, integer pipe 50%, DRAM 55%):
// codes straight into registers, two blocks of 128 k ahead; widened there;
// multiplied by mma.sync with the rows as M = 16 and the tokens as N = 8 or 16
// (the matrix unit is idle most of the time, so its older path is enough);
// group sums scaled and added in fp32.  Of rows g + 8 r (g = lane / 4) lane t =
// lane % 4 of a quad reads the t-th quarter of every group, and its codes
// take the places of the k that the instruction expects in that lane; x
// stands in shared memory in the same order, so nothing is shuffled.  `split`
// warps share a tile's k and add their sums in a fixed order.
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 512;
constexpr int kFewTokens = 16;
constexpr int kFewRows = 32;             // rows of a tile: two M = 16 that share every read of x
constexpr size_t kFewSmem = 224 * 1024;  // x and the split's sums at most

// Bytes of one token of x: its 128-k blocks, and 64 more if needed so that two
// neighbouring tokens lie in different halves of the banks.
__host__ __device__ __forceinline__ int few_pitch(int H) { return (H + 127) / 128 * 256 + 64; }
static size_t few_smem(int M, int H) {   // x, then two sets of sums
    const int NT = (M + 7) / 8;
    return static_cast<size_t>(M) * few_pitch(H) + sizeof(float) * 2 * kFewThreads * NT * 8;
}

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's codes of one group: kWords words.  Groups of 32 and 64 leave part of
// a 32-byte sector to the next load, which finds it in L1.
template <int WORDS> __device__ __forceinline__ void ld_codes(uint32_t *w, const uint8_t *p) {
    if (WORDS == 4) {
        const uint4 u = ld_stream(p);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if (WORDS == 2) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = u.x; w[1] = u.y;
    } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
}

// NT: token tiles of 8.  ZERO: the weights have zero points.
template <int NT, int GROUP, bool ZERO>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(HeadArgs a, int split) {
    constexpr int kSubs = 128 / GROUP, kWords = GROUP / 32, kWarps = kFewThreads / 32;
    constexpr int kAhead = 2;             // blocks on their way
    constexpr int kSet = GROUP == 32 ? kAhead : 2;   // scale sets: one a block, or the current and the next
    extern __shared__ __align__(16) char dyn[];
    __shared__ int rows[kFewTokens];
    __shared__ int s_count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    griddep_wait();
    griddep_launch_dependents();
    if (tid == 0) {
        int n = 0;
        for (int b = 0; b < a.B; ++b)
            for (int p = 0, np = row_positions(a, b); p < np; ++p) rows[n++] = b * a.P + p;
        s_count = n;
    }
    __syncthreads();
    const int count = s_count, pitch = few_pitch(a.H), nkb = (a.H + 127) / 128;
    if (count == 0) return;
    float(*sums)[kWarps][NT * 8][32] = reinterpret_cast<float(*)[kWarps][NT * 8][32]>(dyn + a.B * a.P * pitch);
    // x: chunk (block kb, word w, lane t) of a token at 16 kb + 4 w + t, its eight
    // values in the order 0 4 1 5 2 6 3 7 (see widen8).
    const int per = nkb * 16;
    for (int i = tid; i < count * per; i += kFewThreads) {
        const int tok = i / per, c = i - tok * per;
        uint4 u = make_uint4(0, 0, 0, 0);     // past the end: groups without a share (see live below)
        if (c * 8 < a.H) u = __ldg(reinterpret_cast<const uint4 *>(a.x + static_cast<long long>(rows[tok]) * a.H) + c);
        uint4 w;
        w.x = __byte_perm(u.x, u.z, 0x5410);
        w.y = __byte_perm(u.x, u.z, 0x7632);
        w.z = __byte_perm(u.y, u.w, 0x5410);
        w.w = __byte_perm(u.y, u.w, 0x7632);
        constexpr int kIn = GROUP / 8;    // chunks of a group: kWords for each lane of a quad
        const int q = (c & 15) / kIn, ct = (c & 15) % kIn / kWords, cw = (c & 15) % kWords;
        *reinterpret_cast<uint4 *>(dyn + tok * pitch + ((c & ~15) + (q * kWords + cw) * 4 + ct) * 16) = w;
    }
    __syncthreads();

    // This warp's blocks of a tile's k, and its tiles: the blocks of all of
    // them are one sequence, so the loads run ahead across tiles too.
    const int share = warp % split, lo = nkb * share / split, hi = nkb * (share + 1) / split;
    const int tiles = (a.V + kFewRows - 1) / kFewRows, stride = gridDim.x * (kWarps / split);
    const int first = blockIdx.x * (kWarps / split) + warp / split;
    // The last tile ends with the last row; rows it shares with the one
    // before are computed twice, to the same bits.
    auto tile_row = [&](int tile) { return min(tile * kFewRows, a.V - kFewRows); };
    const long long row_bytes = a.H / 2;
    const char *xb[NT];                   // this lane's tokens and place; columns past the last token are not used
#pragma unroll
    for (int n = 0; n < NT; ++n) xb[n] = dyn + min(8 * n + g, count - 1) * pitch + t * 16;

    // Rows g + 8 r.  Codes on their way; scales and zero points by sets of four
    // groups, of which each lane of a quad holds one: the rows' reads touch a
    // quarter of the lines, and a shuffle hands them on.
    uint32_t w[kAhead][4][4] = {}, sc[kSet][4], zp[kSet][4];
    const uint8_t *codes = nullptr;       // next block to fetch, row g
    long long par = 0;                    // index of its first scale, row g
    int f_tile = first, f_kb = lo;
    auto aim = [&]() {
        const long long v = tile_row(f_tile) + g;
        codes = a.codes + v * row_bytes + lo * 64 + t * (GROUP / 8);
        par = v * a.G + lo * kSubs;
    };
    // The set that was fetched becomes the one at hand.
    auto take_set = [&](int set, int from) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            sc[set][r] = a.scale_f32 ? sc[from][r] : sc[from][r] << 16;
            if (ZERO) zp[set][r] = zero_pair(zp[from][r] & 15u);
        }
    };
    // That is left to the set's first block, whose loads have had the longest,
    // but for a share whose last set has a single block: its set is taken
    // before the next tile's first set is fetched over it.
    bool lone = false;
    auto fetch = [&](int u) {
        if (lone && f_kb == lo) take_set(0, 1);
        if (f_tile >= tiles) return;
#pragma unroll
        for (int q = 0; q < kSubs; ++q) {
            if (kSubs == 1 || f_kb * kSubs + q < a.G)
#pragma unroll
            for (int r = 0; r < 4; ++r) ld_codes<kWords>(w[u][r] + q * kWords, codes + r * 8 * row_bytes + q * (GROUP / 2));
        }
        if ((f_kb - lo) * kSubs % 4 == 0) {
            const int set = GROUP == 32 ? u : 1;
            const int in = min(t, a.G - 1 - f_kb * kSubs);    // past the end: any
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const long long at = par + r * 8ll * a.G + in;
                sc[set][r] = a.scale_f32 ? __ldg(static_cast<const uint32_t *>(a.scale) + at)
                                         : __ldg(static_cast<const unsigned short *>(a.scale) + at);
                if (ZERO) zp[set][r] = __ldg(a.zero + at);
            }
        }
        codes += 64;
        par += kSubs;
        if (++f_kb == hi) {
            f_kb = lo;
            f_tile += stride;
            aim();
        }
    };
    float acc[2][NT][4];
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    };
    // The split's sums of a finished tile.  Two sets in turn: a warp that
    // writes a set has passed the barrier after which its readers were done.
    int turn = 0;
    auto finish = [&](int tile) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[turn][warp][(m * NT + n) * 4 + i][lane] = acc[m][n][i];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / split), "r"(32 * split) : "memory");
        for (int i = share; i < 8 * NT; i += split) {
            float y = 0.f;
            for (int j = 0; j < split; ++j) y += sums[turn][warp - share + j][i][lane];
            y *= 64.f;                    // widen8 gives code / 64
            const int tok = i / 4 % NT * 8 + 2 * t + (i & 1);
            const int v = tile_row(tile) + i / (4 * NT) * 16 + g + (i & 2) * 4;
            if (tok < count) {
                const long long o = static_cast<long long>(rows[tok]) * a.V + v;
                if (a.out_f32) store_logit(static_cast<float *>(a.out) + o, y);
                else store_logit(static_cast<__nv_bfloat16 *>(a.out) + o, y);
            }
        }
        turn ^= 1;
        clear();
    };
    clear();
    if (lo == hi) {                       // more warps than blocks: nothing to add
        for (int tile = first; tile < tiles; tile += stride) finish(tile);
        return;
    }
    aim();
    fetch(0);
    lone = GROUP != 32 && (hi - 1 - lo) * kSubs % 4 == 0;
    static_assert(kAhead == 2, "a set at hand and one on its way");
    fetch(1);
    const uint32_t eight = zero_pair(8);
    int tile = first, kb = lo;
    while (tile < tiles) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int in_set = (kb - lo) * kSubs % 4;     // this block's first group in its set
            const int set = GROUP == 32 ? u : 0;
            if (in_set == 0 && !(lone && kb + 1 == hi)) take_set(set, GROUP == 32 ? u : 1);
            const int xo = kb * 256;
#pragma unroll
            for (int q = 0; q < kSubs; ++q) {
                // No branch here, so that the groups' products overlap.
                const bool live = kSubs == 1 || kb * kSubs + q < a.G;
                const int from = (lane & ~3) + in_set + q;
                float f[4];
                uint32_t o[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    f[r] = __uint_as_float(__shfl_sync(0xffffffffu, sc[set][r], from));
                    if (!live) f[r] = 0.f;
                    o[r] = ZERO ? __shfl_sync(0xffffffffu, zp[set][r], from) : eight;
                }
                float part[2][NT][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) part[m][n][i] = 0.f;
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    uint4 b[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        b[n] = *reinterpret_cast<const uint4 *>(xb[n] + xo + (q * kWords + i) * 64);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t r0[4], r1[4];
                        widen8(w[u][2 * m][q * kWords + i], o[2 * m], r0);
                        widen8(w[u][2 * m + 1][q * kWords + i], o[2 * m + 1], r1);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_16x8x16(part[m][n], r0[0], r1[0], r0[1], r1[1], b[n].x, b[n].y);
                            mma_16x8x16(part[m][n], r0[2], r1[2], r0[3], r1[3], b[n].z, b[n].w);
                        }
                    }
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[m][n][i] = fmaf(f[2 * m + i / 2], part[m][n][i], acc[m][n][i]);
            }
            fetch(u);
            if (++kb == hi) {
                finish(tile);
                kb = lo;
                tile += stride;
                if (tile >= tiles) break;
            }
        }
    }
}

template <int NT, int GROUP, bool ZERO> static cudaError_t launch_few(const HeadArgs &a, int M, cudaStream_t st) {
    static std::atomic<bool> attr_set[64];
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && !attr_set[dev & 63].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(few_kernel<NT, GROUP, ZERO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kFewSmem));
        if (e == cudaSuccess) attr_set[dev & 63].store(true, std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
    // Four warps to a tile keep the last round of tiles short; sixteen where
    // there are too few tiles to occupy the SMs otherwise.
    const int tiles = (a.V + kFewRows - 1) / kFewRows, split = tiles <= 4 * sms ? 16 : 4;
    const int per = kFewThreads / 32 / split, need = (tiles + per - 1) / per;
    return launch_pdl(few_kernel<NT, GROUP, ZERO>, dim3(need < sms ? need : sms), dim3(kFewThreads), few_smem(M, a.H), st,
                      a, split);
}

template <int NT, bool ZERO> static cudaError_t launch_few_group(const HeadArgs &a, int M, cudaStream_t st) {
    if (a.group == 128) return launch_few<NT, 128, ZERO>(a, M, st);
    if (a.group == 64) return launch_few<NT, 64, ZERO>(a, M, st);
    return launch_few<NT, 32, ZERO>(a, M, st);
}

static cudaError_t launch_few_tokens(const HeadArgs &a, int M, cudaStream_t st) {
    if (M <= 8) return a.zero ? launch_few_group<1, true>(a, M, st) : launch_few_group<1, false>(a, M, st);
    return a.zero ? launch_few_group<2, true>(a, M, st) : launch_few_group<2, false>(a, M, st);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
static sv_status head_check(const sv_w4 *w, int B, int P) {
    if (!w) return SV_ERR_ARG;
    if (w->scale_dtype != SV_F32 && w->scale_dtype != SV_BF16) return SV_ERR_DTYPE;
    if (w->V < 1 || w->V > SV_MAX_V || w->H < 1 || w->H > SV_MAX_H ||
        (w->group != 32 && w->group != 64 && w->group != 128) || w->H % w->group)
        return SV_ERR_SHAPE;
    if (B < 0 || P < 1 || static_cast<long long>(B) * P > (1 << 20)) return SV_ERR_SHAPE;
    return SV_OK;
}

// Halves, tokens of each and k per stage, for a batch of at most M tokens.
static int halves_for(int M) { return M <= 128 ? 1 : 2; }
static int nh_for(int M) { return M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 96; }
static int ak_for(int nh) { return nh <= 64 ? 256 : 128; }

static bool few(const sv_w4 *w, int M) {
    return M <= kFewTokens && w->V >= kFewRows && few_smem(M, w->H) <= kFewSmem;
}

// Shares of a row's k: as many as the SMs of a B200 allow beside the tiles (not
// those of the current device: the workspace's size must not depend on it).  The
// longest share must be kSplitSaves stages shorter than the row, or the third
// launch costs more than it saves (20 tokens: 1152 x 1952, groups of 128, one
// stage less 10.7 to 13.1 us; 960 x 2830, groups of 64, two less 12.1 to 12.4 at
// 52 tokens; 1600 x 3000, groups of 32, five less 18.1 to 13.4; 4608 x 2752 19 to
// 13; 336 tokens of 12288 x 1000 185 to 42).  Up to kSplitTokens tokens the
// shares' sums (76 KB a token at most) stay in L2.
constexpr int kSms = 148, kSplitSaves = 3, kSplitTokens = 1024;

static int splits_for(const sv_w4 *w, int M) {
    const int ak = ak_for(nh_for(M)), nkb = (w->H + ak - 1) / ak, G = w->H / w->group, subs = ak / w->group;
    const int tiles = (w->V + kTileV - 1) / kTileV, chunks = (G + kParGroups - 1) / kParGroups;
    const int n = kSms / tiles < chunks ? kSms / tiles : chunks;
    if (n < 2 || M > kSplitTokens) return 1;
    int longest = 0;
    for (int i = 0; i < n; ++i) {
        const int k = span_of(i, n, G, nkb, subs).nkb;
        if (k > longest) longest = k;
    }
    return nkb - longest >= kSplitSaves ? n : 1;
}

struct HeadPlan {
    size_t off_rows, off_image, off_part, bytes;
    int splits;
};

static HeadPlan head_plan(const sv_w4 *w, int B, int P) {
    const int M = B * P, nh = nh_for(M), ak = ak_for(nh), nkb = (w->H + ak - 1) / ak;
    HeadPlan p;
    auto align = [](size_t o) { return (o + 1023) & ~static_cast<size_t>(1023); };
    p.off_rows = 16;
    p.off_image = align(16 + 4ull * M);
    // Whatever the scheduled count is, it packs into at most as many passes
    // as M does, each of at most that many tokens.
    const size_t most = halves_for(M) * nh, passes = (M + most - 1) / most;
    p.off_part = align(p.off_image + passes * most * nkb * ak * 2ull);
    p.splits = splits_for(w, M);
    const size_t tiles = (w->V + kTileV - 1) / kTileV;
    p.bytes = p.off_part + (p.splits > 1 ? p.splits * M * tiles * kTileV * sizeof(float) : 0);
    return p;
}

// The codes as a two-dimensional tensor of bytes, in tiles of 128 rows of one
// stage; what lies past the matrix reads as 0.
static cudaError_t code_map(const sv_w4 *w, int ak, CUtensorMap *map) {
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                               const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<Encode> encode{nullptr};
    Encode f = encode.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
        f = reinterpret_cast<Encode>(p);
        encode.store(f, std::memory_order_release);
    }
    const cuuint64_t dim[2] = {static_cast<cuuint64_t>(w->H / 2), static_cast<cuuint64_t>(w->V)};
    const cuuint64_t stride[1] = {static_cast<cuuint64_t>(w->H / 2)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(ak / 2), kTileV}, step[2] = {1, 1};
    const CUresult r = f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(w->codes), dim, stride, box, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE,
                         ak == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int HALVES, int NH, int GROUP>
static cudaError_t launch_head(const HeadArgs &a, const CUtensorMap &map, cudaStream_t st) {
    using Cfg = HeadCfg<HALVES, NH, GROUP>;
    static std::atomic<bool> attr_set[64];
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && !attr_set[dev & 63].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(head_kernel<HALVES, NH, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
        if (e == cudaSuccess) attr_set[dev & 63].store(true, std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(head_kernel<HALVES, NH, GROUP>, dim3(a.splits > 1 ? a.splits * a.tiles : a.tiles < sms ? a.tiles : sms), dim3(Cfg::kThreads), Cfg::kSmem,
                      st, a, map);
}

template <int HALVES, int NH> static cudaError_t launch_group(const HeadArgs &a, const CUtensorMap &map, cudaStream_t st) {
    if (a.group == 128) return launch_head<HALVES, NH, 128>(a, map, st);
    if (a.group == 64) return launch_head<HALVES, NH, 64>(a, map, st);
    return launch_head<HALVES, NH, 32>(a, map, st);
}

}  // namespace sv

extern "C" size_t sv_head_w4_workspace_bytes(const sv_w4 *weight, int B, int P) {
    if (sv::head_check(weight, B, P) != SV_OK || B == 0 || sv::few(weight, B * P)) return 0;
    // Enough for every smaller batch too: up to kSplitTokens tokens there may be
    // sums of shares, which larger batches do without.
    const size_t own = sv::head_plan(weight, B, P).bytes;
    const size_t split = B * P > sv::kSplitTokens ? sv::head_plan(weight, sv::kSplitTokens, 1).bytes : 0;
    return own > split ? own : split;
}

extern "C" sv_status sv_head_w4(const sv_w4 *weight, const void *x, int B, int P,
                                const int32_t *lengths, int extra, void *out, sv_dtype out_dtype,
                                void *workspace, size_t workspace_bytes, int32_t *status,
                                void *stream) {
    sv::NvtxRange nvtx_range("sv_head_w4");
    if (const sv_status e = sv::head_check(weight, B, P)) return e;
    if (out_dtype != SV_F32 && out_dtype != SV_BF16) return SV_ERR_DTYPE;
    if (B == 0) return SV_OK;
    if (!weight->codes || !weight->scale || !x || !out) return SV_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(weight->codes) | reinterpret_cast<uintptr_t>(x) |
         reinterpret_cast<uintptr_t>(workspace)) & 15)
        return SV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(weight->scale) & (weight->scale_dtype == SV_F32 ? 3 : 1)) return SV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(out) & (out_dtype == SV_F32 ? 3 : 1)) return SV_ERR_ARG;
    if (sv::misaligned4(lengths, status)) return SV_ERR_ARG;
    const bool few = sv::few(weight, B * P);
    if (!few && !workspace) return SV_ERR_ARG;
    const sv::HeadPlan p = sv::head_plan(weight, B, P);
    if (!few && workspace_bytes < p.bytes) return SV_ERR_WORKSPACE;
    sv::HeadArgs a = {};
    a.codes = weight->codes; a.scale = weight->scale; a.zero = weight->zero;
    a.scale_f32 = weight->scale_dtype == SV_F32;
    a.out_f32 = out_dtype == SV_F32;
    a.V = weight->V; a.H = weight->H; a.group = weight->group; a.G = weight->H / weight->group;
    a.tiles = (a.V + sv::kTileV - 1) / sv::kTileV;
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.B = B; a.P = P; a.lengths = lengths; a.extra = extra; a.out = out;
    const int M = B * P;
    if (few)
        return sv::note_cuda(sv::launch_few_tokens(a, M, static_cast<cudaStream_t>(stream)));
    a.halves = sv::halves_for(M);
    a.nh_max = sv::nh_for(M);
    a.ak = sv::ak_for(a.nh_max);
    a.nkb = (a.H + a.ak - 1) / a.ak;
    char *w = static_cast<char *>(workspace);
    a.count = reinterpret_cast<int *>(w);
    a.rows = reinterpret_cast<int *>(w + p.off_rows);
    a.image = w + p.off_image;
    a.splits = p.splits;
    a.part = reinterpret_cast<float *>(w + p.off_part);
    a.status = status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int packs = M < sv::kPackGrid ? M : sv::kPackGrid;
    cudaError_t e = sv::launch_pdl(sv::pack_kernel, dim3(packs), dim3(sv::kPackThreads), 0, st, a);
    if (e != cudaSuccess) return sv::note_cuda(e);
    // After a launch, which makes the device's context this thread's: the
    // driver's call needs one, and a new host thread has none.
    CUtensorMap map;
    e = sv::code_map(weight, a.ak, &map);
    if (e != cudaSuccess) return sv::note_cuda(e);
    switch (a.nh_max) {
    case 32: e = sv::launch_group<1, 32>(a, map, st); break;
    case 64: e = sv::launch_group<1, 64>(a, map, st); break;
    case 128: e = sv::launch_group<1, 128>(a, map, st); break;
    default: e = sv::launch_group<2, 96>(a, map, st); break;
    }
    if (e == cudaSuccess && a.splits > 1)
        e = sv::launch_pdl(sv::join_kernel, dim3(M, (a.V + 4 * sv::kJoinThreads - 1) / (4 * sv::kJoinThreads)),
                           dim3(sv::kJoinThreads), 0, st, a);
    return sv::note_cuda(e);
}
