// Products grouped by expert for few rows per expert (decode and small batches),
// on the warp-level tensor instructions; lq_grouped.cu routes here.
//
//   z[i][r] = s[r] sum_k sigma[r][k] u[row(i)][k] + bias[r]
//
// The weights are read once per pass of at most 8 NT columns and bound the kernel,
// so the contraction is arranged around them: signs become the A operand of
// mma.sync m16n8k16 (bf16, fp32 accumulate), 16 weight rows by 16 k, and up to 8
// rows of u are its 8 columns. +-1 and u are exact in bf16, so only the fp32 sums
// round; NaN and Inf propagate as IEEE sums do.
//
// A block is 16 H weight rows by one pass of one expert; blocks go round the
// CTAs (one per SM). K is walked in runs of 1024 (32 sign words). Four producer
// warps copy a run's words [16 H][32] and its slice of u's rows [cols][1024] into
// a ring of shared-memory stages with cp.async (16-byte pieces; 8 or 4 bytes where
// a row of words is not 16-byte aligned), zeros past K and past the last row. Eight
// consumer warps are two groups of four that take alternate runs; the four warps of a
// group take a quarter of the run each (8 words, 256 k) of all 16 H rows. A warp
// keeps its u fragments of the run in registers while it walks the rows, so each
// sign word is expanded once and each u fragment loaded once per 16 H rows.
// At the end of a block the eight warps' sums are added in warp order through
// shared memory (the result does not depend on timing), and the epilogue runs.
//
// Order of k. Thread (g, t) = (lane / 4, lane % 4) owns words t and 4 + t of the
// warp's eight. Register j of a word holds bits j and j + 16 at the sign positions
// of a bf16 pair, one shift and one logic operation per two weights:
// ((w << (15 - j)) & 0x80008000) ^ 0xBF80BF80. The matching u pair (k, k + 16) is
// picked from two 16-byte loads. Threads with t >= 2 load the upper half of a word's u
// first, which keeps the eight lanes of a load phase on different banks; their
// words are rotated by 16 to match.
#include "lq_debug.cuh"
#include "lq_epilogue.cuh"
#include "lq_grouped.cuh"
#include "lq_internal.h"
#include "lq_sm100.cuh"

namespace lq {
namespace {

using namespace sm100;

constexpr int kRunWords = 32, kRunK = 1024;  // one stage of K
constexpr int kConsumers = 8, kProducers = 4;
constexpr int kThreads = 32 * (kConsumers + kProducers);
constexpr int kUPitch = kRunK * 2 + 16;  // bytes of one u row of a stage: 16 off a multiple of 32
constexpr int kMaxStages = 16;
constexpr size_t kSmemMax = 227 * 1024 - 1024;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
template <int B>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(B), "r"(there ? B : 0)
                 : "memory");
}
// Arrives on the barrier once every earlier cp.async of this thread has landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

struct Plan {
    uint32_t shift[16];  // 2^(15 - j): kept from the compiler, so that it multiplies (see sign_pair)
    int stages, stage_bytes, cols_cap, cols_pass, nblk;
    int planes;  // columns per slot: 1, or 3 bf16 parts of an fp32 u
    size_t smem;
};

// Bits j and j + 16 of w as a pair of bf16 +-1. The shift is written as a product
// with a kernel argument: an integer multiply-add runs on the FMA pipe beside the
// logic operation on the ALU pipe, and the ALU pipe (half a warp instruction per
// clock) bounded the kernel with both on it.
__device__ __forceinline__ uint32_t sign_pair(uint32_t w, const Plan& p, int j) {
    const uint32_t x = j == 15 ? w : w * p.shift[j];
    uint32_t r;  // (x & b) ^ c in one instruction
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(x), "r"(0x80008000u), "r"(0xBF80BF80u));
    return r;
}

template <int H, int NT, int VEC>
__global__ void __launch_bounds__(kThreads, 1) mma_kernel(const __grid_constant__ GroupedCall c, const __grid_constant__ Plan p, unsigned* status) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int R = 16 * H, RP = R + 4, COLS = 8 * NT;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 16 * kMaxStages);
    float* red = reinterpret_cast<float*>(smem + 512);  // [8 warps][COLS][RP]
    const uint32_t ring = smem_addr(smem) + 512 + kConsumers * COLS * RP * 4;
    const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * kMaxStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kw = c.K >> 5, runs = (kw + kRunWords - 1) / kRunWords;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(full0 + 8 * i, 32 * kProducers);
            mbar_init(empty0 + 8 * i, 4);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();

    UnitWalk walk;
    Unit u;
    const int per = p.cols_pass / p.planes;  // slots of a unit
    int st = 0, phase = 0;
    if (warp >= kConsumers) {
        // ---- producers
        const int tid = threadIdx.x - 32 * kConsumers;
        bool stop = false;  // the same in all lanes of a warp
        for (long long unit = blockIdx.x; !stop && walk.find<true>(c, per, p.nblk, unit, lane, u); unit += gridDim.x) {
            const int e = u.e, slot0 = u.slot0, slots = u.slots, row0 = u.blk * R, cols = slots * p.planes;
            const uint32_t* w0 = c.packed + ((long long)e * c.out + row0) * kw;
            const int rows_left = c.out - row0;
            for (int run = 0; run < runs; ++run) {
                const bool free = !*abort_flag && mbar_wait(empty0 + 8 * st, phase ^ 1, status);
                if (!__all_sync(0xffffffffu, free)) {
                    *abort_flag = 1;
                    stop = true;
                    break;
                }
                const uint32_t a_st = ring + st * p.stage_bytes, u_st = a_st + R * 128;
                const int word0 = run * kRunWords;
                // sign words: piece x of row r goes to 16-byte chunk (x / 16) ^ (r % 8) of the row
                constexpr int PIECES = 128 / VEC;
                for (int i = tid; i < R * PIECES; i += 32 * kProducers) {
                    const int r = i / PIECES, x = (i % PIECES) * (VEC / 4);
                    const bool there = r < rows_left && word0 + x < kw &&
                                       LQ_IN_BOUNDS(((long long)e * c.out + row0 + r) * kw + word0 + x + VEC / 4 - 1,
                                                    (long long)c.experts * c.out * kw);
                    const uint32_t dst = a_st + r * 128 + (((x >> 2) ^ (r & 7)) << 4) + (x & 3) * 4;
                    const void* src = there ? w0 + (long long)r * kw + word0 + x : c.packed;
                    if constexpr (VEC == 16)
                        cp_async16(dst, src, there);
                    else
                        cp_async_small<VEC>(dst, src, there);
                }
                // u rows of the columns
                for (int i = tid; i < cols * (kRunK / 8); i += 32 * kProducers) {
                    const int col = i >> 7, x = (i & 127) * 8;
                    const int slot = slot0 + col / p.planes;
                    long long row = c.rows ? (long long)__ldg(c.rows + slot) : slot;
                    bool there = row >= 0 && row < c.tokens && run * kRunK + x < c.K;
                    row = row * p.planes + col % p.planes;
                    there = there && LQ_IN_BOUNDS(row * c.K + run * kRunK + x + 7, (long long)c.tokens * p.planes * c.K);
                    const uint16_t* ub = static_cast<const uint16_t*>(c.u);
                    cp_async16(u_st + col * kUPitch + x * 2, there ? ub + row * c.K + run * kRunK + x : ub, there);
                }
                cp_async_arrive(full0 + 8 * st);
                if (++st == p.stages) st = 0, phase ^= 1;
            }
        }
        cp_async_wait_all();
        return;
    }

    // ---- consumers
    const int g = lane >> 2, t = lane & 3, quarter = warp & 3, group = warp >> 2;
    const uint32_t rot = t >= 2 ? 0x1032u : 0x3210u;
    long long done = 0;  // runs before this unit, over all units
    for (long long unit = blockIdx.x; walk.find<true>(c, per, p.nblk, unit, lane, u); unit += gridDim.x) {
        const int e = u.e, slot0 = u.slot0, slots = u.slots, row0 = u.blk * R, cols = slots * p.planes;
        float acc[H][NT][4];
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][n][j] = 0.f;
        for (int run = 0; run < runs; ++run) {
            const bool mine = ((done + run) & 1) == group;
            if (mine) {
                if (!*abort_flag && !mbar_wait(full0 + 8 * st, phase, status)) *abort_flag = 1;
                const uint32_t a_st = ring + st * p.stage_bytes;
                const uint32_t u_st = a_st + R * 128 + quarter * 512 + t * 64 + (t >= 2 ? 32 : 0);
                const uint32_t u_other = t >= 2 ? -32 : 32;
                uint32_t b[NT][2][16];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int col = 8 * n + g;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
                            if (col < cols) {
                                const uint32_t at = u_st + col * kUPitch + x * 256 + h * 16;
                                lo = lds128(at);
                                hi = lds128(at + u_other);
                            }
                            const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, v[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                b[n][x][8 * h + 2 * i] = __byte_perm(l[i], v[i], 0x5410);
                                b[n][x][8 * h + 2 * i + 1] = __byte_perm(l[i], v[i], 0x7632);
                            }
                        }
                }
                // row g of tile i: chunk 2 quarter + x, swizzled by the row; rows 8 apart share the swizzle
                const uint32_t a_row = a_st + g * 128 + t * 4;
#pragma unroll
                for (int i = 0; i < H; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t at = a_row + i * 2048 + (((2 * quarter + x) ^ g) << 4);
                        const uint32_t wl = __byte_perm(lds32(at), 0, rot), wh = __byte_perm(lds32(at + 1024), 0, rot);
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const uint32_t a0 = sign_pair(wl, p, j), a1 = sign_pair(wh, p, j);
                            const uint32_t a2 = sign_pair(wl, p, j + 1), a3 = sign_pair(wh, p, j + 1);
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_bf16(acc[i][n], a0, a1, a2, a3, b[n][x][j], b[n][x][j + 1]);
                        }
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * st);
            }
            if (++st == p.stages) st = 0, phase ^= 1;
        }
        done += runs;

        // ---- the warps' sums, in warp order
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    red[(warp * COLS + 8 * n + 2 * t + (j & 1)) * RP + 16 * i + g + (j >> 1) * 8] = acc[i][n][j];
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (!*abort_flag) {
            const int step = c.glu ? 2 : 1, per_col = R / step, width = c.glu ? c.out / 2 : c.out;
            for (int x = threadIdx.x; x < slots * per_col; x += 32 * kConsumers) {
                const int slot = x / per_col, r = (x - slot * per_col) * step;
                if (row0 + r >= c.out) continue;
                float z[2] = {0.f, 0.f};
                for (int q = 0; q < p.planes; ++q)
                    for (int w = 0; w < kConsumers; ++w)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (h < step) z[h] += red[(w * COLS + slot * p.planes + q) * RP + r + h];
                for (int h = 0; h < step; ++h) {
                    const long long at = (long long)e * c.out + row0 + r + h;
                    z[h] = __ldg(c.s + at) * z[h] + (c.bias ? __ldg(c.bias + at) : 0.f);
                }
                const float y = c.glu ? activate(z[0], c.act) * z[1] : activate(z[0], c.act);
                const long long at = (long long)(slot0 + slot) * width + (row0 + r) / step;
                if (LQ_IN_BOUNDS(at, (long long)c.n * width))
                    store_elem(c.o, at, c.o_bf16, c.residual ? y + load_elem(c.residual, at, c.o_bf16) : y);
            }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
    }
}

// fp32 u as three bf16 parts that add up to it exactly (24 significant bits, cut
// toward zero so that nothing overflows): row 3 b + p of the planes is part p of row
// b. NaN and Inf stay in the first part.
__global__ void split_kernel(const float* __restrict__ u, long long count, int K, uint16_t* __restrict__ planes) {
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < count; i += (long long)gridDim.x * blockDim.x) {
        const float v = __ldg(u + i);
        const uint32_t bits = __float_as_uint(v);
        uint32_t hi = bits & 0xFFFF0000u, mid = 0, lo = 0;
        if ((bits & 0x7F800000u) != 0x7F800000u) {
            const float rest = v - __uint_as_float(hi);
            mid = __float_as_uint(rest) & 0xFFFF0000u;
            lo = __float_as_uint(rest - __uint_as_float(mid));
        } else if (bits & 0x007FFFFFu) {
            hi |= 0x00400000u;  // a NaN stays one
        }
        const long long b = i / K, k = i - b * K;
        planes[(3 * b) * K + k] = (uint16_t)(hi >> 16);
        planes[(3 * b + 1) * K + k] = (uint16_t)(mid >> 16);
        planes[(3 * b + 2) * K + k] = (uint16_t)(lo >> 16);
    }
}

template <int H, int NT, int VEC>
cudaError_t launch_vec(const GroupedCall& c, const Plan& p, unsigned* status, cudaStream_t st, int sms) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(mma_kernel<H, NT, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    mma_kernel<H, NT, VEC><<<sms, kThreads, p.smem, st>>>(c, p, status);
    return cudaGetLastError();
}

template <int H, int NT>
cudaError_t launch_h(const GroupedCall& c, Plan p, unsigned* status, cudaStream_t st, int sms) {
    const size_t head = 512 + (size_t)kConsumers * 8 * NT * (16 * H + 4) * 4;
    p.stage_bytes = 16 * H * 128 + (p.cols_cap * kUPitch + 127) / 128 * 128;
    p.nblk = (c.out + 16 * H - 1) / (16 * H);
    p.stages = (int)((kSmemMax - head) / p.stage_bytes);
    p.stages = p.stages > kMaxStages ? kMaxStages : p.stages;
    p.smem = head + (size_t)p.stages * p.stage_bytes;
    const int kw = c.K >> 5;
    if (kw % 4 == 0) return launch_vec<H, NT, 16>(c, p, status, st, sms);
    if (kw % 2 == 0) return launch_vec<H, NT, 8>(c, p, status, st, sms);
    return launch_vec<H, NT, 4>(c, p, status, st, sms);
}

}  // namespace

size_t grouped_mma_workspace_size(int K, int n, bool u_bf16) {
    return u_bf16 ? 0 : (size_t)3 * n * K * 2;
}

cudaError_t launch_grouped_mma(const GroupedCall& call, void* ws, unsigned* status, cudaStream_t st, int sms) {
    GroupedCall c = call;
    Plan p{};
    p.planes = c.u_bf16 ? 1 : 3;
    for (int j = 0; j < 16; ++j) p.shift[j] = 1u << (15 - j);
    if (!c.u_bf16) {
        const long long count = (long long)c.tokens * c.K;
        split_kernel<<<(int)((count + 255) / 256 < 4 * sms ? (count + 255) / 256 : 4 * sms), 256, 0, st>>>(
            static_cast<const float*>(c.u), count, c.K, static_cast<uint16_t*>(ws));
        c.u = ws;
    }
    // expected slots of an expert that has any: the pass width, 8 or 16 columns
    const int active = c.n < c.experts ? c.n : c.experts;
    const long long each = ((long long)c.n + active - 1) / active * p.planes;
    const int nt = each > 8 ? 2 : 1;
    p.cols_pass = 8 * nt / p.planes * p.planes;
    p.cols_cap = (long long)c.n * p.planes < p.cols_pass ? c.n * p.planes : p.cols_pass;
    // block height: rounds of blocks over the SMs times their length (a block's fixed cost is about one tile)
    const long long tiles = (c.out + 15) / 16, passes = (each + p.cols_pass - 1) / p.cols_pass;
    int best = 1;
    long long best_cost = -1;
    for (int h = 1; h <= (nt == 1 ? 8 : 6); ++h) {
        if (nt == 2 && h == 5) continue;
        const long long units = active * passes * ((tiles + h - 1) / h);
        const long long cost = (units + sms - 1) / sms * (h + 1);
        if (best_cost < 0 || cost < best_cost) best = h, best_cost = cost;
    }
    if (nt == 1) switch (best) {
        case 1: return launch_h<1, 1>(c, p, status, st, sms);
        case 2: return launch_h<2, 1>(c, p, status, st, sms);
        case 3: return launch_h<3, 1>(c, p, status, st, sms);
        case 4: return launch_h<4, 1>(c, p, status, st, sms);
        case 5: return launch_h<5, 1>(c, p, status, st, sms);
        case 6: return launch_h<6, 1>(c, p, status, st, sms);
        case 7: return launch_h<7, 1>(c, p, status, st, sms);
        default: return launch_h<8, 1>(c, p, status, st, sms);
    }
    switch (best) {
        case 1: return launch_h<1, 2>(c, p, status, st, sms);
        case 2: return launch_h<2, 2>(c, p, status, st, sms);
        case 3: return launch_h<3, 2>(c, p, status, st, sms);
        case 4: return launch_h<4, 2>(c, p, status, st, sms);
        default: return launch_h<6, 2>(c, p, status, st, sms);
    }
}

}  // namespace lq

LQ_DEBUG_FLAG_TAKE(debug_take_grouped_mma)
