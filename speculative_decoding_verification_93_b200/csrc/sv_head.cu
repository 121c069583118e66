// sv_head.cu -- output head with 4-bit weights and group scales on the
// tensor cores (tcgen05; the formula stands at sv_head_w4 in include/sv.h).
//
// The product is computed transposed: D[v, token] = sum_k W[v, k] x[token, k]
// with 128 vocabulary rows as the matrix unit's M and the tokens as its N,
// so that few tokens waste little and every weight is read once.
//
// Exactness.  code - zero is an integer of at most five bits, exact in bf16,
// and so is its product with a bf16 x in fp32.  The scale is not folded into
// the bf16 operand (that would round every weight to 8 bits); instead each
// group's sum is read back from tensor memory, multiplied by its scale in
// fp32 and added to fp32 accumulators in registers.
//
// One launch packs the scheduled tokens of x into the operand layout
// (pack_kernel); the second (head_kernel) is persistent, one CTA per SM, and
// walks 128-row tiles of the vocabulary, K in stages of 128:
//   warp 0      copies the stage's x image into a ring of shared memory
//               (bulk copies, mbarrier completion);
//   warps 2, 3  fetch scales and zero points into a ring of their own;
//   one or two warpgroups own one weight row per thread: codes arrive
//               through a ring of asynchronous 16-byte copies, are widened to
//               bf16 integers and written to tensor memory as the A operand;
//   warp 1      issues tcgen05.mma, A from tensor memory, B from shared
//               memory, one batch per (group, half of the tokens);
//   two warpgroups, one per half of the tokens, read each finished batch
//               back, scale and accumulate it, and write the logits.
// The two halves alternate, so the matrix unit works on one half while the
// other is read back.  A in tensor memory keeps the widened weights (four
// times the bytes of the codes) out of shared memory, whose bandwidth the B
// operand needs.
#include <atomic>
#include <climits>
#include <cstdint>

#include "sv.h"
#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

// ---------------------------------------------------------------------------
// Layout shared by both kernels.
// ---------------------------------------------------------------------------
constexpr int kStageK = 128;             // k per stage
constexpr int kTileV = 128;              // vocabulary rows per tile

// Tokens are taken in `passes` of `per` tokens, each pass in `halves` of `nh`
// (a multiple of 16) tokens.  The x image of (pass, stage) holds, per half,
// two blocks of nh rows x 64 k in the 128-byte swizzle.
struct TokenPlan {
    int count, passes, per, halves, nh;
};

__host__ __device__ __forceinline__ TokenPlan token_plan(int count, int nh_max) {
    TokenPlan p;
    p.count = count;
    p.passes = (count + 2 * nh_max - 1) / (2 * nh_max);
    const int share = p.passes ? (count + p.passes - 1) / p.passes : 0;
    p.halves = share <= 16 ? 1 : 2;
    p.nh = p.halves == 1 ? 16 : (share + 31) / 32 * 16;
    p.per = p.halves * p.nh;
    return p;
}

struct HeadArgs {
    const uint8_t *codes;
    const void *scale;
    const uint8_t *zero;
    bool scale_f32, out_f32;
    int V, H, group, G, nkb, tiles;
    const __nv_bfloat16 *x;
    int B, P;
    const int32_t *lengths;
    int extra;
    void *out;
    int nh_max;
    int *count;          // workspace: scheduled tokens
    int *rows;           // workspace [B * P]: output row of each packed token
    char *image;         // workspace: x images
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
    const TokenPlan t = token_plan(run, a.nh_max);
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
        const int kb = c / 16, sub = (c / 8) & 1, col = c & 7;
        char *d = a.image + (static_cast<long long>(pass) * a.nkb + kb) * t.per * 256 +
                  (half * 2 + sub) * t.nh * 128 + r * 128 + ((col ^ (r & 7)) * 16);
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
// D (fp32, tensor memory) (+)= A (bf16, tensor memory) * B (bf16, shared memory)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)) : "memory");
}
// `bar` completes one arrival when every mma issued so far has finished.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&f)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]),
          "=f"(f[8]), "=f"(f[9]), "=f"(f[10]), "=f"(f[11]), "=f"(f[12]), "=f"(f[13]), "=f"(f[14]), "=f"(f[15])
        : "r"(addr) : "memory");
}
// Loads from tensor memory land by the wait; naming their registers here
// keeps every use behind it.
__device__ __forceinline__ void tc_wait_ld(float (&f)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3]), "+f"(f[4]), "+f"(f[5]), "+f"(f[6]), "+f"(f[7]),
                   "+f"(f[8]), "+f"(f[9]), "+f"(f[10]), "+f"(f[11]), "+f"(f[12]), "+f"(f[13]), "+f"(f[14]), "+f"(f[15])
                 :: "memory");
}
template <int N> __device__ __forceinline__ void regs_less() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups
// 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) |
           (2ull << 61);
}

// ---------------------------------------------------------------------------
// 3. The product.
// ---------------------------------------------------------------------------
constexpr int kStageBytes = kTileV * kStageK / 2;   // codes of one stage
constexpr int kASlots = 4;               // A operands in tensor memory: 64 columns each
constexpr int kACol = 256;               // behind the accumulators
constexpr uint32_t kTmemCols = 512;
constexpr int kParGroups = 8;            // groups per chunk of the parameter ring
constexpr int kParSlots = 3;
constexpr uint64_t kHeadWaitNs = 1000000000ull;

// Scale and zero point of kParGroups groups of a tile's rows.  `off` is the
// pair -zero / 64 in bf16 (see widen8).
struct ParChunk {
    float scale[kParGroups][kTileV];
    uint32_t off[kParGroups][kTileV];
};

// Per instantiation: up to NH tokens a half, DB accumulators per half, XS
// stages of x, CS stages of codes, WW warpgroups that widen codes.
// One warpgroup widens a stage in about 400 cycles (latency; 200 of issue),
// the copies of a stage's codes take 350, and the matrix unit 8 nh cycles:
// above 64 tokens a half one is enough, and the accumulators need the
// registers of the second.
template <int NH> struct HeadCfg {
    static constexpr int DB = NH <= 16 ? 4 : NH <= 64 ? 2 : 1;
    static constexpr int XS = NH <= 16 ? 8 : NH <= 64 ? 3 : 2;
    static constexpr int CS = NH <= 64 ? 12 : 8;
    static constexpr int WW = NH <= 64 ? 2 : 1;
    static constexpr int kThreads = 128 * (3 + WW);
    // Registers a thread of the service, widening and accumulating
    // warpgroups: their sum stays below what the CTA was launched with.
    static constexpr int kRegs0 = 56, kRegsW = WW == 2 ? 80 : 88, kRegsA = WW == 2 ? 128 : 184;
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static_assert(kRegs0 + WW * kRegsW + 2 * kRegsA <= (3 + WW) * kLaunchRegs, "register split");
    static constexpr int kXBytes = 2 * NH * 256;
    // At least half of the SM's shared memory: two CTAs on one SM would
    // wait for each other's tensor memory.
    static constexpr int kUsed = 1024 + XS * kXBytes + CS * kStageBytes +
                                 kParSlots * static_cast<int>(sizeof(ParChunk));
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static_assert(CS % WW == 0 && 2 * NH * DB <= kACol && kSmem <= 227 * 1024 - 1024, "head layout");
};

struct HeadBars {
    uint64_t xfull[8], xempty[8];
    uint64_t afull[kASlots], aempty[kASlots];
    uint64_t dfull[8], dempty[8];
    uint64_t pfull[kParSlots], pempty[kParSlots];
    uint64_t drain;
    uint32_t tmem;
};

// A warp-wide bounded wait: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, kHeadWaitNs));
}

__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
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

// The x images of every stage into shared memory (one lane of warp 0).
template <int NH>
__device__ bool copy_role(const HeadArgs &a, const TokenPlan &t, int jobs, HeadBars &bar, char *xring) {
    using Cfg = HeadCfg<NH>;
    const uint32_t bytes = t.per * 256;
    bool ok = true;
    int s = 0;
    for (int job = 0; ok && job < jobs; ++job) {
        const char *src = a.image + static_cast<long long>(job % t.passes) * a.nkb * bytes;
        for (int kb = 0; kb < a.nkb; ++kb, ++s) {
            const int slot = s % Cfg::XS;
            if (!mbar_wait(&bar.xempty[slot], ((s / Cfg::XS) & 1) ^ 1, kHeadWaitNs)) { ok = false; break; }
            mbar_arrive_expect_tx(&bar.xfull[slot], bytes);
            bulk_g2s(xring + slot * Cfg::kXBytes, src + static_cast<long long>(kb) * bytes, bytes, &bar.xfull[slot]);
        }
    }
    // The copies in flight land before this CTA may leave.
    for (int q = max(0, s - Cfg::XS); q < s; ++q)
        mbar_wait(&bar.xfull[q % Cfg::XS], (q / Cfg::XS) & 1, kHeadWaitNs);
    return ok;
}

// The matrix unit's instructions (warp 1: every lane runs the loops, so that
// the operands stay in uniform registers; one lane issues).
template <int NH, int GROUP>
__device__ bool mma_role(const HeadArgs &a, const TokenPlan &t, int jobs, HeadBars &bar, const char *xring,
                         uint32_t tmem) {
    using Cfg = HeadCfg<NH>;
    constexpr int kSubs = kStageK / GROUP;
    const uint32_t nh = warp_value(t.nh);
    const int halves = warp_value(t.halves), stages = warp_value(jobs) * a.nkb;
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((nh >> 3) << 17) | ((kTileV >> 4) << 24);
    const uint64_t x0 = smem_desc(smem_u32(xring));
    const bool issuer = elect_one();
    int i = 0, kb = 0;                    // group (counts through all jobs), stage of the job
    bool ok = true;
    for (int s = 0; s < stages; ++s) {
        const int ab = s % kASlots, slot = s % Cfg::XS;
        if (!warp_wait(&bar.afull[ab], (s / kASlots) & 1) ||
            !warp_wait(&bar.xfull[slot], (s / Cfg::XS) & 1)) { ok = false; break; }
        const int subs = min(kSubs, (a.H - kb * kStageK) / GROUP);
        const uint64_t xs = x0 + static_cast<uint64_t>(slot * (Cfg::kXBytes / 16));
        const uint32_t acol = tmem + kACol + ab * 64;
#pragma unroll
        for (int g = 0; g < kSubs; ++g) {
            if (g >= subs) break;
            for (int h = 0; h < halves; ++h) {
                const int db = h * Cfg::DB + i % Cfg::DB;
                if (!warp_wait(&bar.dempty[db], ((i / Cfg::DB) & 1) ^ 1)) { ok = false; break; }
                tc_fence_after();
                if (issuer) {
                    const uint64_t xh = xs + static_cast<uint64_t>(h * 2 * nh * 8);
#pragma unroll
                    for (int q = 0; q < GROUP / 16; ++q) {
                        const int k16 = g * (GROUP / 16) + q;
                        mma_ts(tmem + db * NH, acol + 8 * k16, xh + (k16 >> 2) * nh * 8 + (k16 & 3) * 2, idesc, q > 0);
                    }
                    mma_commit(&bar.dfull[db]);
                }
                __syncwarp();
            }
            if (!ok) break;
            ++i;
        }
        if (!ok) break;
        if (issuer) {
            mma_commit(&bar.aempty[ab]);
            mma_commit(&bar.xempty[slot]);
        }
        __syncwarp();
        if (++kb == a.nkb) kb = 0;
    }
    // Nothing of the matrix unit is in flight when tensor memory is freed.
    if (issuer) mma_commit(&bar.drain);
    __syncwarp();
    warp_wait(&bar.drain, 0);
    return ok;
}

// Scales and zero points (warps 2 and 3, two rows a lane): as fp32 and bf16
// pairs in shared memory, eight groups at a time, so that the rows' strided
// reads are 16 bytes wide where the alignment allows it, made once for both
// halves, and far ahead of their use.
__device__ bool param_role(const HeadArgs &a, const TokenPlan &t, int jobs, HeadBars &bar, ParChunk *ring) {
    const int l = threadIdx.x & 63;       // warps 2 and 3
    const bool wide = !a.scale_f32 && a.G % 8 == 0 && (reinterpret_cast<uintptr_t>(a.scale) & 15) == 0;
    int c = 0;
    for (int job = 0; job < jobs; ++job) {
        const int tile = blockIdx.x + job / t.passes * gridDim.x;
        for (int g0 = 0; g0 < a.G; g0 += kParGroups, ++c) {
            float sc[2][kParGroups];
            uint32_t zp[2][kParGroups];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const long long at = static_cast<long long>(min(tile * kTileV + r * 64 + l, a.V - 1)) * a.G + g0;
                if (wide) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.scale) + at));
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) { sc[r][2 * q] = bf16_lo(w[q]); sc[r][2 * q + 1] = bf16_hi(w[q]); }
                } else {
#pragma unroll
                    for (int q = 0; q < kParGroups; ++q) {
                        const long long e = at + min(q, a.G - 1 - g0);
                        sc[r][q] = a.scale_f32 ? __ldg(static_cast<const float *>(a.scale) + e)
                                               : ld_elem<2>(static_cast<const char *>(a.scale), e);
                    }
                }
                if (a.zero) {
#pragma unroll
                    for (int q = 0; q < kParGroups; ++q) zp[r][q] = __ldg(a.zero + at + min(q, a.G - 1 - g0)) & 15u;
                }
            }
            ParChunk &p = ring[c % kParSlots];
            if (!warp_wait(&bar.pempty[c % kParSlots], ((c / kParSlots) & 1) ^ 1)) return false;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int q = 0; q < kParGroups; ++q) {
                    p.scale[q][r * 64 + l] = 64.f * sc[r][q];
                    if (a.zero) p.off[q][r * 64 + l] = zero_pair(zp[r][q]);
                }
            mbar_arrive(&bar.pfull[c % kParSlots]);
        }
    }
    return true;
}

// One warpgroup of wi = 0 .. WW - 1: the stages s = wi mod WW, one weight row a
// thread.  Codes come by asynchronous 16-byte copies, four lanes a row (64
// contiguous bytes), each warp for its own 32 rows.
template <int NH, int GROUP> struct Widen {
    using Cfg = HeadCfg<NH>;
    static constexpr int kRing = Cfg::CS / Cfg::WW;   // slots of this warpgroup
    static constexpr int kSubs = kStageK / GROUP;
    const HeadArgs &a;
    char *mine;                           // this warp's rows of the warpgroup's first slot
    int lane, quarter, wi;
    int f_kb, f_pass, f_tile, f_n;        // next stage to fetch, stages fetched
    const uint8_t *src[4];                // this lane's rows in the tile being fetched

    __device__ Widen(const HeadArgs &args, char *ring, int wi_) : a(args), wi(wi_) {
        lane = threadIdx.x & 31;
        quarter = (threadIdx.x >> 5) & 3;
        mine = ring + wi * kRing * kStageBytes + quarter * 32 * 64;
        f_kb = wi; f_pass = 0; f_tile = blockIdx.x; f_n = 0;
        aim();
    }
    __device__ __forceinline__ void aim() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long v = min(f_tile * kTileV + quarter * 32 + 8 * i + (lane >> 2), a.V - 1);
            src[i] = a.codes + v * (a.H / 2) + (lane & 3) * 16;
        }
    }
    // 32-code pieces of stage kb.
    __device__ __forceinline__ int pieces(int kb) const { return min(4, a.H / 32 - 4 * kb); }
    __device__ __forceinline__ void copy() {
        char *slot = mine + (f_n % kRing) * kStageBytes;
        if ((lane & 3) < pieces(f_kb)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + (lane >> 2);
                cp_async16(slot + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) * 16), src[i] + f_kb * 64);
            }
        }
        ++f_n;
        f_kb += Cfg::WW;
    }
    // The first stages of the first tile, whatever the token count.
    __device__ void start() {
#pragma unroll 1
        for (int i = 0; i < kRing - 1; ++i) {
            if (f_kb < a.nkb) copy();
            cp_async_commit();
        }
    }
    __device__ bool run(const TokenPlan &t, int jobs, HeadBars &bar, const ParChunk *par, uint32_t tmem) {
        const int stages = jobs * a.nkb;
        int to_fetch = (stages - wi + Cfg::WW - 1) / Cfg::WW;
        int kb = wi, c0 = 0;              // stage of the job; chunks of the jobs before it
        const int chunks = (a.G + kParGroups - 1) / kParGroups;
        int have = -1;                    // chunk of the parameter ring at hand
        // start() left kRing - 1 groups, some perhaps empty: fill up in order.
        int n = 0;                        // stages of this warpgroup done
        auto fetch = [&]() {
            if (f_n < to_fetch) {
                while (f_kb >= a.nkb) {
                    f_kb -= a.nkb;
                    if (++f_pass == t.passes) { f_pass = 0; f_tile += gridDim.x; aim(); }
                }
                copy();
            }
            cp_async_commit();
        };
        // Where the first tile had too few stages for the ring, restart the
        // count: later groups complete later, so waiting by count stays right.
        const int lead = f_n;             // stages in flight (<= kRing - 1)
        for (int i = lead; i < kRing - 1; ++i) fetch();
        for (int s = wi; s < stages; s += Cfg::WW, ++n) {
            cp_async_wait<kRing - 2>();
            __syncwarp();                 // every lane's copies of the stage have landed
            fetch();
            while (kb >= a.nkb) { kb -= a.nkb; c0 += chunks; }
            const char *row = mine + (n % kRing) * kStageBytes + lane * 64;
            const int np = pieces(kb);
            uint32_t off[kSubs];
            if (a.zero) {
#pragma unroll
                for (int g = 0; g < kSubs; ++g) {
                    const int gi = min(kb * kSubs + g, a.G - 1), c = c0 + gi / kParGroups;
                    while (have < c) {    // hand back the chunks behind it, wait for the next
                        if (have >= 0) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar.pempty[have % kParSlots]);
                        }
                        ++have;
                        if (!warp_wait(&bar.pfull[have % kParSlots], (have / kParSlots) & 1)) return false;
                    }
                    off[g] = par[c % kParSlots].off[gi % kParGroups][quarter * 32 + lane];
                }
            } else {
#pragma unroll
                for (int g = 0; g < kSubs; ++g) off[g] = zero_pair(8);
            }
            const int ab = s % kASlots;
            if (!warp_wait(&bar.aempty[ab], ((s / kASlots) & 1) ^ 1)) return false;
            tc_fence_after();
            const uint32_t dst = tmem + kACol + ab * 64 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (2 * h >= np) break;
                uint32_t r[32];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int pc = 2 * h + j;
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (pc < np) u = *reinterpret_cast<const uint4 *>(row + ((pc ^ ((lane >> 1) & 3)) * 16));
                    const uint32_t o = off[pc * 32 / GROUP];
                    widen8(u.x, o, r + j * 16);
                    widen8(u.y, o, r + j * 16 + 4);
                    widen8(u.z, o, r + j * 16 + 8);
                    widen8(u.w, o, r + j * 16 + 12);
                }
                tmem_st32(dst + h * 32, r);
            }
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(&bar.afull[ab]);
            kb += Cfg::WW;
        }
        // Chunks that this warpgroup had no stage in (or its last ones).
        if (a.zero) {
            const int all = jobs * chunks;
            for (; have < all; ++have) {
                if (have >= 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.pempty[have % kParSlots]);
                }
                if (have + 1 < all && !warp_wait(&bar.pfull[(have + 1) % kParSlots], ((have + 1) / kParSlots) & 1))
                    return false;
            }
        }
        return true;
    }
};

// One warpgroup per half of the tokens; a thread owns one vocabulary row.
template <int NH>
__device__ bool accumulate_role(const HeadArgs &a, const TokenPlan &t, int jobs, HeadBars &bar,
                                const ParChunk *par, uint32_t tmem, int h) {
    using Cfg = HeadCfg<NH>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    int i = 0, c = 0;
    for (int job = 0; job < jobs; ++job) {
        const int tile = blockIdx.x + job / t.passes * gridDim.x, pass = job % t.passes;
        const int v = tile * kTileV + quarter * 32 + lane;
        float acc[NH];
#pragma unroll
        for (int n = 0; n < NH; ++n) acc[n] = 0.f;
        for (int g0 = 0; g0 < a.G; g0 += kParGroups, ++c) {
            const int slot = c % kParSlots, ng = min(kParGroups, a.G - g0);
            if (!warp_wait(&bar.pfull[slot], (c / kParSlots) & 1)) return false;
            for (int q = 0; q < ng; ++q, ++i) {
                const float sc = par[slot].scale[q][quarter * 32 + lane];
                const float2 ss = make_float2(sc, sc);
                const int db = h * Cfg::DB + i % Cfg::DB;
                if (!warp_wait(&bar.dfull[db], (i / Cfg::DB) & 1)) return false;
                tc_fence_after();
                const uint32_t src = lanes + db * NH;
                // The next 16 columns are on their way while these are added.
                float d[2][16];
                tmem_ld16(src, d[0]);
#pragma unroll
                for (int k = 0; k < NH / 16; ++k) {
                    if (16 * k < t.nh) {
                        tc_wait_ld(d[k & 1]);
                        if (k + 1 < NH / 16 && 16 * (k + 1) < t.nh) tmem_ld16(src + 16 * (k + 1), d[(k + 1) & 1]);
#pragma unroll
                        for (int n = 0; n < 16; n += 2) {
                            float *y = acc + 16 * k + n;
                            const float2 z = __ffma2_rn(make_float2(d[k & 1][n], d[k & 1][n + 1]), ss, make_float2(y[0], y[1]));
                            y[0] = z.x;
                            y[1] = z.y;
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(&bar.dempty[db]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.pempty[slot]);
        }
        // One vocabulary row per lane: a warp writes 32 consecutive logits of each token.
        const int t0 = pass * t.per + h * t.nh, live = min(t.nh, t.count - t0);
#pragma unroll
        for (int n0 = 0; n0 < NH; n0 += 8) {
            if (n0 < live) {
                int row[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) row[n] = __ldg(a.rows + t0 + min(n0 + n, live - 1));
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    if (n0 + n < live && v < a.V) {
                        const long long at = static_cast<long long>(row[n]) * a.V + v;
                        if (a.out_f32) static_cast<float *>(a.out)[at] = acc[n0 + n];
                        else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(acc[n0 + n]);
                    }
                }
            }
        }
    }
    return true;
}

template <int NH, int GROUP>
__global__ void __launch_bounds__(HeadCfg<NH>::kThreads, 1) head_kernel(HeadArgs a) {
    using Cfg = HeadCfg<NH>;
    extern __shared__ char dyn[];
    __shared__ HeadBars bar;
    char *xring = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    char *cring = xring + Cfg::XS * Cfg::kXBytes;
    ParChunk *par = reinterpret_cast<ParChunk *>(cring + Cfg::CS * kStageBytes);
    const int tid = threadIdx.x, warp = warp_value(tid >> 5), lane = tid & 31, wg = warp >> 2;
    // The codes of the first stages are asked for at once: the pack kernel
    // let this grid launch after its own wait, so whatever ran before this
    // call has finished.
    Widen<NH, GROUP> widen(a, cring, wg >= 1 && wg <= Cfg::WW ? wg - 1 : 0);
    if (wg >= 1 && wg <= Cfg::WW) widen.start();
    if (warp == 0) tmem_alloc(&bar.tmem, kTmemCols);
    if (warp == 1 && lane == 0) {
        for (int i = 0; i < Cfg::XS; ++i) { mbar_init(&bar.xfull[i], 1); mbar_init(&bar.xempty[i], 1); }
        for (int i = 0; i < kASlots; ++i) { mbar_init(&bar.afull[i], 128); mbar_init(&bar.aempty[i], 1); }
        for (int i = 0; i < 2 * Cfg::DB; ++i) { mbar_init(&bar.dfull[i], 1); mbar_init(&bar.dempty[i], 128); }
        mbar_init(&bar.drain, 1);
    }
    griddep_wait();
    griddep_launch_dependents();
    const TokenPlan t = token_plan(__ldcg(a.count), a.nh_max);
    if (warp == 1 && lane == 0) {
        for (int i = 0; i < kParSlots; ++i) {
            mbar_init(&bar.pfull[i], 64);
            mbar_init(&bar.pempty[i], 4 * t.halves + (a.zero ? 4 * Cfg::WW : 0));
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = warp_value(bar.tmem);
    const int my_tiles = (a.tiles - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
                         static_cast<int>(gridDim.x);
    const int jobs = my_tiles * t.passes;
    bool ok = true;
    if (wg == 0) {
        regs_less<Cfg::kRegs0>();
        if (warp == 0) {
            if (lane == 0) ok = copy_role<NH>(a, t, jobs, bar, xring);
        } else if (warp == 1) {
            ok = mma_role<NH, GROUP>(a, t, jobs, bar, xring, tmem);
        } else {
            ok = param_role(a, t, jobs, bar, par);
        }
    } else if (wg <= Cfg::WW) {
        regs_less<Cfg::kRegsW>();
        ok = widen.run(t, jobs, bar, par, tmem);
        cp_async_wait<0>();
    } else {
        regs_more<Cfg::kRegsA>();
        const int h = wg - 1 - Cfg::WW;
        if (h < t.halves) ok = accumulate_role<NH>(a, t, jobs, bar, par, tmem, h);
    }
    if (!ok && a.status) atomicOr(a.status, SV_NOTE_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free(tmem, kTmemCols);
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

// Tokens per half for a batch of at most M tokens.
static int nh_for(int M) { return M <= 32 ? 16 : M <= 128 ? 64 : 128; }

struct HeadPlan {
    size_t off_rows, off_image, bytes;
};

static HeadPlan head_plan(const sv_w4 *w, int B, int P) {
    const int M = B * P, nh = nh_for(M), nkb = (w->H + kStageK - 1) / kStageK;
    HeadPlan p;
    auto align = [](size_t o) { return (o + 1023) & ~static_cast<size_t>(1023); };
    p.off_rows = 16;
    p.off_image = align(16 + 4ull * M);
    // Whatever the scheduled count is, it packs into as many passes as M at
    // most, each of at most 2 nh tokens.
    const size_t passes = (M + 2 * nh - 1) / (2 * nh);
    p.bytes = p.off_image + passes * 2 * nh * nkb * 256ull;
    return p;
}

template <int NH, int GROUP>
static cudaError_t launch_head(const HeadArgs &a, cudaStream_t st) {
    static std::atomic<bool> attr_set[64];
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && !attr_set[dev & 63].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(head_kernel<NH, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 HeadCfg<NH>::kSmem);
        if (e == cudaSuccess) attr_set[dev & 63].store(true, std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(head_kernel<NH, GROUP>, dim3(a.tiles < sms ? a.tiles : sms), dim3(HeadCfg<NH>::kThreads),
                      HeadCfg<NH>::kSmem, st, a);
}

template <int NH> static cudaError_t launch_group(const HeadArgs &a, cudaStream_t st) {
    if (a.group == 128) return launch_head<NH, 128>(a, st);
    if (a.group == 64) return launch_head<NH, 64>(a, st);
    return launch_head<NH, 32>(a, st);
}

}  // namespace sv

extern "C" size_t sv_head_w4_workspace_bytes(const sv_w4 *weight, int B, int P) {
    if (sv::head_check(weight, B, P) != SV_OK || B == 0) return 0;
    return sv::head_plan(weight, B, P).bytes;
}

extern "C" sv_status sv_head_w4(const sv_w4 *weight, const void *x, int B, int P,
                                const int32_t *lengths, int extra, void *out, sv_dtype out_dtype,
                                void *workspace, size_t workspace_bytes, int32_t *status,
                                void *stream) {
    sv::NvtxRange nvtx_range("sv_head_w4");
    if (const sv_status e = sv::head_check(weight, B, P)) return e;
    if (out_dtype != SV_F32 && out_dtype != SV_BF16) return SV_ERR_DTYPE;
    if (B == 0) return SV_OK;
    if (!weight->codes || !weight->scale || !x || !out || !workspace) return SV_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(weight->codes) | reinterpret_cast<uintptr_t>(x) |
         reinterpret_cast<uintptr_t>(workspace)) & 15)
        return SV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(weight->scale) & (weight->scale_dtype == SV_F32 ? 3 : 1)) return SV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(out) & (out_dtype == SV_F32 ? 3 : 1)) return SV_ERR_ARG;
    const sv::HeadPlan p = sv::head_plan(weight, B, P);
    if (workspace_bytes < p.bytes) return SV_ERR_WORKSPACE;
    sv::HeadArgs a = {};
    a.codes = weight->codes; a.scale = weight->scale; a.zero = weight->zero;
    a.scale_f32 = weight->scale_dtype == SV_F32;
    a.out_f32 = out_dtype == SV_F32;
    a.V = weight->V; a.H = weight->H; a.group = weight->group; a.G = weight->H / weight->group;
    a.nkb = (a.H + sv::kStageK - 1) / sv::kStageK;
    a.tiles = (a.V + sv::kTileV - 1) / sv::kTileV;
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.B = B; a.P = P; a.lengths = lengths; a.extra = extra; a.out = out;
    const int M = B * P;
    a.nh_max = sv::nh_for(M);
    char *w = static_cast<char *>(workspace);
    a.count = reinterpret_cast<int *>(w);
    a.rows = reinterpret_cast<int *>(w + p.off_rows);
    a.image = w + p.off_image;
    a.status = status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int packs = M < sv::kPackGrid ? M : sv::kPackGrid;
    cudaError_t e = sv::launch_pdl(sv::pack_kernel, dim3(packs), dim3(sv::kPackThreads), 0, st, a);
    if (e != cudaSuccess) return sv::note_cuda(e);
    switch (a.nh_max) {
    case 16: e = sv::launch_group<16>(a, st); break;
    case 64: e = sv::launch_group<64>(a, st); break;
    default: e = sv::launch_group<128>(a, st); break;
    }
    return sv::note_cuda(e);
}
