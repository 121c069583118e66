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
//   warps 4-7   own one weight row per thread: codes arrive through a ring of
//               asynchronous 16-byte copies, are widened to bf16 integers
//               (one logic operation and one exact subtraction for two
//               codes) and written to tensor memory as the A operand;
//   warp 1      one thread issues tcgen05.mma, A from tensor memory, B from
//               shared memory, one batch per (group, half of the tokens);
//   warps 8-15  one warpgroup per half of the tokens reads each finished
//               batch back, scales and accumulates it, and writes the logits.
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
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
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
constexpr int kHeadThreads = 512;
constexpr int kCodeSlots = 8;            // ring of code stages: 8 KB each
constexpr int kASlots = 4;               // A operands in tensor memory: 64 columns each
constexpr int kACol = 256;               // behind the accumulators
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kHeadWaitNs = 1000000000ull;

// Per instantiation: up to NH tokens a half, DB accumulators per half, XS
// stages of x.
template <int NH> struct HeadCfg {
    static constexpr int DB = NH <= 64 ? 2 : 1;
    static constexpr int XS = NH <= 16 ? 8 : NH <= 64 ? 4 : 2;
    static constexpr int kXBytes = 2 * NH * 256;
    static constexpr int kCodeBytes = kCodeSlots * kTileV * 64;
    static constexpr int kUsed = 1024 + XS * kXBytes + kCodeBytes;
    // At least half of the SM's shared memory: two CTAs on one SM would
    // wait for each other's tensor memory.
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
};

struct HeadBars {
    uint64_t xfull[8], xempty[8];
    uint64_t afull[kASlots], aempty[kASlots];
    uint64_t dfull[4], dempty[4];
    uint64_t drain;
    uint32_t tmem;
};

// A warp-wide bounded wait: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, kHeadWaitNs));
}

__device__ __forceinline__ float ld_scale(const HeadArgs &a, long long at) {
    return a.scale_f32 ? __ldg(static_cast<const float *>(a.scale) + at)
                       : ld_elem<2>(static_cast<const char *>(a.scale), at);
}

// Eight codes to four pairs of bf16 integers: 128 + code by one logic
// operation (the ulp of bf16 in [128, 256) is 1), minus 128 + zero, exact.
__device__ __forceinline__ void widen8(uint32_t w, __nv_bfloat162 off, uint32_t *r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&p), off);
        r[i] = *reinterpret_cast<const uint32_t *>(&d);
    }
}

// Warps 4-7.  GROUP is the weights' group.
template <int GROUP>
__device__ bool widen_role(const HeadArgs &a, HeadBars &bar, char *ring, uint32_t tmem, int passes) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    char *mine = ring + quarter * 32 * 64;              // this warp's 32 rows of a slot
    constexpr int kSlot = kTileV * 64;
    const long long row_bytes = a.H / 2;
    const int tail_pieces = ((a.H % kStageK) ? (a.H % kStageK) : kStageK) / 32;
    const int my_tiles = (a.tiles - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
                         static_cast<int>(gridDim.x);
    const int total = my_tiles * passes * a.nkb;   // stages of this CTA
    int f_kb = 0, f_pass = 0, f_tile = blockIdx.x, f_s = 0;   // next stage to fetch
    auto fetch = [&]() {
        if (f_s < total) {
            char *slot = mine + (f_s % kCodeSlots) * kSlot;
            const int pieces = f_kb == a.nkb - 1 ? tail_pieces : 4;
            const int j = lane & 3;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + (lane >> 2);
                const long long v = min(f_tile * kTileV + quarter * 32 + r, a.V - 1);
                if (j < pieces)
                    cp_async16(slot + r * 64 + ((j ^ ((r >> 1) & 3)) * 16),
                               a.codes + v * row_bytes + f_kb * 64 + j * 16);
            }
            ++f_s;
            if (++f_kb == a.nkb) {
                f_kb = 0;
                if (++f_pass == passes) { f_pass = 0; f_tile += gridDim.x; }
            }
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kCodeSlots - 1; ++i) fetch();
    int kb = 0, pass = 0, tile = blockIdx.x;
    for (int s = 0; s < total; ++s) {
        cp_async_wait<kCodeSlots - 2>();
        __syncwarp();          // every lane's copies of stage s have landed; stage s - 1 is read
        fetch();
        const long long v = min(tile * kTileV + quarter * 32 + lane, a.V - 1);
        const char *row = mine + (s % kCodeSlots) * kSlot + lane * 64;
        const int pieces = kb == a.nkb - 1 ? tail_pieces : 4;
        constexpr int kSubs = kStageK / GROUP;
        __nv_bfloat162 off[kSubs];
#pragma unroll
        for (int g = 0; g < kSubs; ++g) {
            uint32_t z = 8;
            if (a.zero) z = __ldg(a.zero + v * a.G + min(kb * kSubs + g, a.G - 1)) & 15u;
            const uint32_t o = 0x43004300u | (z * 0x00010001u);
            off[g] = *reinterpret_cast<const __nv_bfloat162 *>(&o);
        }
        const int ab = s % kASlots;
        if (!warp_wait(&bar.aempty[ab], ((s / kASlots) & 1) ^ 1)) return false;
        tc_fence_after();
        const uint32_t dst = tmem + kACol + ab * 64 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (2 * h >= pieces) break;
            uint32_t r[32];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int pc = 2 * h + j;
                uint4 u = make_uint4(0, 0, 0, 0);
                if (pc < pieces) u = *reinterpret_cast<const uint4 *>(row + ((pc ^ ((lane >> 1) & 3)) * 16));
                const __nv_bfloat162 o = off[pc * 32 / GROUP];
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
        if (++kb == a.nkb) {
            kb = 0;
            if (++pass == passes) { pass = 0; tile += gridDim.x; }
        }
    }
    return true;
}

template <int NH, int GROUP>
__global__ void __launch_bounds__(kHeadThreads, 1) head_kernel(HeadArgs a) {
    using Cfg = HeadCfg<NH>;
    constexpr int DB = Cfg::DB, XS = Cfg::XS, kSubs = kStageK / GROUP;
    extern __shared__ char dyn[];
    __shared__ HeadBars bar;
    char *xring = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    char *cring = xring + XS * Cfg::kXBytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = tid >> 7;
    if (tid == 0) {
        for (int i = 0; i < XS; ++i) { mbar_init(&bar.xfull[i], 1); mbar_init(&bar.xempty[i], 1); }
        for (int i = 0; i < kASlots; ++i) { mbar_init(&bar.afull[i], 128); mbar_init(&bar.aempty[i], 1); }
        for (int i = 0; i < 4; ++i) { mbar_init(&bar.dfull[i], 1); mbar_init(&bar.dempty[i], 128); }
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&bar.tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    griddep_wait();
    griddep_launch_dependents();
    const TokenPlan t = token_plan(__ldcg(a.count), a.nh_max);
    const int my_tiles = (a.tiles - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
                         static_cast<int>(gridDim.x);
    const int jobs = my_tiles * t.passes;
    bool ok = true;

    if (wg == 0) {
        regs_less<56>();
        if (warp == 0 && lane == 0) {
            const uint32_t bytes = t.per * 256;
            int s = 0;
            for (int job = 0; ok && job < jobs; ++job) {
                const char *src = a.image + static_cast<long long>(job % t.passes) * a.nkb * bytes;
                for (int kb = 0; kb < a.nkb; ++kb, ++s) {
                    const int slot = s % XS;
                    if (!mbar_wait(&bar.xempty[slot], ((s / XS) & 1) ^ 1, kHeadWaitNs)) { ok = false; break; }
                    mbar_arrive_expect_tx(&bar.xfull[slot], bytes);
                    bulk_g2s(xring + slot * Cfg::kXBytes, src + static_cast<long long>(kb) * bytes, bytes,
                             &bar.xfull[slot]);
                }
            }
            // The copies in flight land before this CTA may leave.
            for (int q = max(0, s - XS); q < s; ++q)
                mbar_wait(&bar.xfull[q % XS], (q / XS) & 1, kHeadWaitNs);
        } else if (warp == 1 && lane == 0) {
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((t.nh >> 3) << 17) | ((kTileV >> 4) << 24);
            int s = 0, i = 0;             // stage, group (both count through all jobs)
            for (int job = 0; ok && job < jobs; ++job) {
                for (int kb = 0; ok && kb < a.nkb; ++kb, ++s) {
                    const int ab = s % kASlots, slot = s % XS;
                    if (!mbar_wait(&bar.afull[ab], (s / kASlots) & 1, kHeadWaitNs) ||
                        !mbar_wait(&bar.xfull[slot], (s / XS) & 1, kHeadWaitNs)) { ok = false; break; }
                    tc_fence_after();
                    const int subs = min(kSubs, (a.H - kb * kStageK) / GROUP);
                    const uint32_t xs = smem_u32(xring + slot * Cfg::kXBytes);
                    const uint32_t acol = tmem + kACol + ab * 64;
                    for (int g = 0; ok && g < subs; ++g, ++i) {
                        for (int h = 0; h < t.halves; ++h) {
                            const int db = h * DB + i % DB;
                            if (!mbar_wait(&bar.dempty[db], ((i / DB) & 1) ^ 1, kHeadWaitNs)) { ok = false; break; }
                            tc_fence_after();
#pragma unroll
                            for (int q = 0; q < GROUP / 16; ++q) {
                                const int k16 = g * (GROUP / 16) + q;
                                const uint32_t b = xs + (h * 2 + (k16 >> 2)) * t.nh * 128 + (k16 & 3) * 32;
                                mma_ts(tmem + db * NH, acol + 8 * k16, smem_desc(b), idesc, q > 0);
                            }
                            mma_commit(&bar.dfull[db]);
                        }
                    }
                    if (ok) {
                        mma_commit(&bar.aempty[ab]);
                        mma_commit(&bar.xempty[slot]);
                    }
                }
            }
            // Nothing of the matrix unit is in flight when tensor memory is freed.
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, kHeadWaitNs);
        }
    } else if (wg == 1) {
        regs_less<96>();
        ok = widen_role<GROUP>(a, bar, cring, tmem, t.passes);
        cp_async_wait<0>();
    } else {
        regs_more<176>();
        const int h = wg - 2, quarter = warp & 3;
        if (h < t.halves) {
            const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            int i = 0;
            for (int job = 0; ok && job < jobs; ++job) {
                const int tile = blockIdx.x + job / t.passes * gridDim.x, pass = job % t.passes;
                const int v = tile * kTileV + quarter * 32 + lane;
                const long long srow = static_cast<long long>(min(v, a.V - 1)) * a.G;
                float acc[NH];
#pragma unroll
                for (int n = 0; n < NH; ++n) acc[n] = 0.f;
                float next = ld_scale(a, srow);
                for (int g = 0; g < a.G; ++g, ++i) {
                    const float sc = next;
                    next = ld_scale(a, srow + min(g + 1, a.G - 1));
                    const int db = h * DB + i % DB;
                    if (!warp_wait(&bar.dfull[db], (i / DB) & 1)) { ok = false; break; }
                    tc_fence_after();
                    const float2 ss = make_float2(sc, sc);
#pragma unroll
                    for (int c = 0; c < NH; c += 16) {
                        if (c < t.nh) {
                            float d[16];
                            tmem_ld16(lanes + db * NH + c, d);
                            tc_wait_ld();
#pragma unroll
                            for (int n = 0; n < 16; n += 2) {
                                const float2 y = __ffma2_rn(make_float2(d[n], d[n + 1]), ss,
                                                            make_float2(acc[c + n], acc[c + n + 1]));
                                acc[c + n] = y.x;
                                acc[c + n + 1] = y.y;
                            }
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(&bar.dempty[db]);
                }
                if (!ok) break;
                // One vocabulary row per lane: a warp writes 32 consecutive logits of each token.
                const int t0 = pass * t.per + h * t.nh;
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    if (n < t.nh && t0 + n < t.count && v < a.V) {
                        const long long at = static_cast<long long>(__ldg(a.rows + t0 + n)) * a.V + v;
                        if (a.out_f32) static_cast<float *>(a.out)[at] = acc[n];
                        else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(acc[n]);
                    }
                }
            }
        }
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
    return launch_pdl(head_kernel<NH, GROUP>, dim3(a.tiles < sms ? a.tiles : sms), dim3(kHeadThreads),
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
