// Products grouped by expert for few rows per expert (decode and small batches),
// on the warp-level tensor instructions; lq_grouped.cu routes here.
//
//   z[i][r] = s[r] sum_k sigma[r][k] u[row(i)][k] + bias[r]
//
// The weights are read once per pass of at most 8 columns and bound the kernel,
// so the contraction is arranged around them: signs become the A operand of
// mma.sync m16n8k16 (bf16, fp32 accumulate), 16 weight rows by 16 k, and rows of u
// are its columns. +-1 and u are exact in bf16, so only the fp32 sums round; NaN and Inf
// propagate as IEEE sums do.
//
// A block is up to H tiles of 16 weight rows by one pass of one expert; blocks go round the
// CTAs (one per SM). K is walked in runs of 1024 (32 sign words) through a ring of
// shared-memory stages. Four producer warps fill them, each every fourth run: the block's
// words of the run [16 h][32] by TMA (128-byte swizzle; 4-byte cp.async in the same layout
// where rows of words are not 16-byte aligned) and the run's slice of u's rows [cols][1024] by
// cp.async, zeros past K. Eight consumer warps form two groups that take the runs in turn; the four
// warps of a group take a quarter of the run each (8 words, 256 k) of all rows. A warp keeps its
// u fragments of the run in registers while it walks the rows, so each sign word is expanded
// once and each u fragment loaded once per 16 h rows. At the end of a block the warps leave their
// sums in shared memory and go on; four warps of their own add them in warp order (the result
// does not depend on timing) and run the epilogue.
//
// What bounds it: the expansion. An MMA takes eight clocks of the tensor pipe of a scheduler, the four
// shifts and four logic operations of its signs eight of the half-rate integer and logic pipes each,
// and ~20 clocks are measured: 20 us for 8 tokens of 13824 x 12288 (1.06 TB/s of signs), 54 us for 8 gated tokens of
// 28672 x 20480 (1.36 TB/s).
//
// Order of k. Thread (g, t) = (lane / 4, lane % 4) owns words t and 4 + t of the
// warp's eight. Register j of a word holds bits j and j + 16 at the sign positions
// of a bf16 pair, one shift and one logic operation per two weights:
// ((w << (15 - j)) & 0x80008000) ^ 0xBF80BF80. The matching u pair (k, k + 16) is
// picked from two 16-byte loads. Threads with t >= 2 load the upper half of a word's u
// first, which keeps the eight lanes of a load phase on different banks; their
// words are rotated by 16 to match.
#include <cuda.h>

#include "lq_debug.cuh"
#include "lq_epilogue.cuh"
#include "lq_grouped.cuh"
#include "lq_internal.h"
#include "lq_sm100.cuh"

namespace lq {
namespace {

using namespace sm100;

constexpr int kRunWords = 32, kRunK = 1024;  // one stage of K
constexpr int kProducers = 4;                // warps
constexpr int kUPitch = kRunK * 2 + 16;      // bytes of one u row of a stage: 16 off a multiple of 32
constexpr int kMaxStages = 16;
constexpr size_t kSmemMax = 227 * 1024 - 2048;
static_assert(kProducers % 2 == 0, "stages in rounds of the producers are whole rounds of the two groups");
constexpr size_t kHead = 512 + 512;  // barriers, zeros

constexpr int COLS = 8, H = 8;  // columns of a pass, tiles of 16 rows that a block may have
// Two groups of consumers: a third (registers moved over from the other warps) changed no time by more than 2%.
constexpr int GROUPS = 2, CONSUMERS = 4 * GROUPS, EPILOGUE = CONSUMERS + kProducers, THREADS = 32 * (EPILOGUE + 4);

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
// Arrives on the barrier once every earlier cp.async of this thread has landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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
// One lane of a converged warp, in the form that lets the compiler keep the operands of
// the instructions behind it in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

struct Plan {
    uint32_t shift[16];  // 2^(15 - j): kept from the compiler, so that it multiplies (see sign_pair)
    int stages, stage_bytes, rp;    // rp: pitch of a column of the warps' sums, in floats
    int nblk, hmax;                 // blocks of an expert's rows; a block has hmax tiles or one less
    int tall, low;                  // the first `tall` blocks have low + 1 tiles, the others low
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

// First tile and number of tiles of block blk: the tiles cut evenly.
__device__ __forceinline__ int block_tiles(const Plan& p, int blk, int& tile0) {
    tile0 = blk * p.low + min(blk, p.tall);
    return p.low + (blk < p.tall);
}

// TMA: rows of sign words are 16-byte aligned and come by TMA.
template <bool TMA>
__global__ void __launch_bounds__(THREADS, 1)
    mma_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap wmap_less,
               const __grid_constant__ GroupedCall c, const __grid_constant__ Plan p, unsigned* status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);  // for the 128-byte swizzle
    const uint32_t ring = smem_addr(smem);
    uint8_t* tail = smem + p.stages * p.stage_bytes;
    const uint32_t full0 = smem_addr(tail), empty0 = full0 + 8 * kMaxStages;
    const uint32_t red_full = full0 + 16 * kMaxStages, red_empty = red_full + 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 16 * kMaxStages + 16);
    const uint32_t zeros = smem_addr(tail + 512);
    float* red = reinterpret_cast<float*>(tail + kHead);  // [consumers][COLS][rp]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kw = c.K >> 5, runs = (kw + kRunWords - 1) / kRunWords;

    if (threadIdx.x < 128) reinterpret_cast<uint32_t*>(tail + 512)[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(full0 + 8 * i, 32 + (TMA ? 1 : 0));
            mbar_init(empty0 + 8 * i, 4);
        }
        mbar_init(red_full, CONSUMERS);
        mbar_init(red_empty, 4);
        *abort_flag = 0;
        fence_barrier_init();
        if (TMA) {
            prefetch_tensormap(&wmap);
            prefetch_tensormap(&wmap_less);
        }
    }
    __syncthreads();

    UnitWalk walk;
    Unit u;
    int st = 0, phase = 0;
    auto advance = [&] {
        if (++st == p.stages) st = 0, phase ^= 1;
    };
    if (warp >= EPILOGUE) {
        // ---- epilogue of a block, while the consumers are at the next one: the warps' sums in warp order
        // A thread owns one output row of the block (a pair of weight rows when gated) and every per-th slot of the pass.
        const int step = c.glu ? 2 : 1, width = c.glu ? c.out / 2 : c.out, tid = threadIdx.x - 32 * EPILOGUE;
        for (long long unit = blockIdx.x; walk.find<true>(c, COLS, p.nblk, unit, lane, u); unit += gridDim.x) {
            int tile0;
            const int h = block_tiles(p, u.blk, tile0), outputs = 16 * h / step, per = 128 / outputs;
            const int first = tid / outputs, r = (tid - first * outputs) * step, row = 16 * tile0 + r;
            const bool mine = first < per && row < c.out;
            float scale[2] = {0.f, 0.f}, shift[2] = {0.f, 0.f};  // before the sums are there
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (mine && i < step) {
                    const long long at = (long long)u.e * c.out + row + i;
                    scale[i] = __ldg(c.s + at);
                    if (c.bias) shift[i] = __ldg(c.bias + at);
                }
            if (!mbar_try_wait(red_full, phase) && !*abort_flag && !mbar_wait(red_full, phase, status)) *abort_flag = 1;
            constexpr int MANY = 4;  // outputs of a thread at a time
            for (int slot0 = first; mine && slot0 < u.slots && !*abort_flag; slot0 += MANY * per) {
                float y[MANY], other[MANY], res[MANY];
                const long long at0 = (long long)(u.slot0 + slot0) * width + row / step, at_step = (long long)per * width;
#pragma unroll
                for (int m = 0; m < MANY; ++m) {
                    const int slot = slot0 + m * per;
                    const bool there = slot < u.slots;
                    res[m] = there && c.residual && LQ_IN_BOUNDS(at0 + m * at_step, (long long)c.n * width) ? load_elem(c.residual, at0 + m * at_step, c.o_bf16) : 0.f;
                    float z[2] = {0.f, 0.f};
                    const float* sums = red + (there ? slot : slot0) * p.rp + r;
                    if (c.glu) {
#pragma unroll
                        for (int w = 0; w < CONSUMERS; ++w) {
                            const float2 v = *reinterpret_cast<const float2*>(sums + w * COLS * p.rp);
                            z[0] += v.x, z[1] += v.y;
                        }
                    } else {
#pragma unroll
                        for (int w = 0; w < CONSUMERS; ++w) z[0] += sums[w * COLS * p.rp];
                    }
                    y[m] = scale[0] * z[0] + shift[0];
                    other[m] = scale[1] * z[1] + shift[1];
                }
                activate_all(y, c.act);
#pragma unroll
                for (int m = 0; m < MANY; ++m) {
                    if (c.glu) y[m] *= other[m];
                    if (c.residual) y[m] += res[m];
                    if (slot0 + m * per < u.slots && LQ_IN_BOUNDS(at0 + m * at_step, (long long)c.n * width))
                        store_elem(c.o, at0 + m * at_step, c.o_bf16, y[m]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(red_empty);
            phase ^= 1;
        }
        return;
    }
    if (warp >= CONSUMERS) {
        // ---- producers: each of the four warps fills every fourth run alone, so that four of these chains of
        // waits and copies run beside one another (one run at a time, a quarter of its copies to a warp, took
        // 550 to 1300 clocks a run and bounded the kernel)
        const int mine = warp - CONSUMERS;
        bool stop = false;  // the same in all lanes of a warp
        int turn = 0, last = -1, last_phase = 0;
        for (long long unit = blockIdx.x; !stop && walk.find<true>(c, COLS, p.nblk, unit, lane, u); unit += gridDim.x) {
            int tile0;
            const int h = block_tiles(p, u.blk, tile0), rows_left = c.out - 16 * tile0;
            const uint16_t* src[COLS];  // this lane's first 16 bytes of each slot's row of u, or null
#pragma unroll
            for (int i = 0; i < COLS; ++i) {
                src[i] = nullptr;
                if (i < u.slots) {
                    const long long row = c.rows ? (long long)__ldg(c.rows + u.slot0 + i) : u.slot0 + i;
                    if (row >= 0 && row < c.tokens) src[i] = c.u + row * c.K + 8 * lane;
                }
            }
            for (int run = 0; run < runs; ++run) {
                const bool own = turn == mine;
                if (++turn == kProducers) turn = 0;
                if (!own) {
                    advance();
                    continue;
                }
                const uint32_t a_st = ring + st * p.stage_bytes, bar = full0 + 8 * st;
                const bool free = mbar_try_wait(empty0 + 8 * st, phase ^ 1) ||
                                  (!*abort_flag && mbar_wait(empty0 + 8 * st, phase ^ 1, status));
                if (!__all_sync(0xffffffffu, free)) {
                    *abort_flag = 1;
                    stop = true;
                    break;
                }
                if (TMA) {
                    if (elect_one()) {
                        mbar_arrive_expect_tx(bar, h * 2048);
                        tma_load_2d(a_st, h == p.hmax ? &wmap : &wmap_less, run * kRunWords, u.e * c.out + 16 * tile0, bar);
                    }
                    __syncwarp();
                } else {
                    // word x of row r goes to 16-byte chunk (x / 4) ^ (r % 8) of the row, as TMA would put it
                    const uint32_t* w0 = c.packed + ((long long)u.e * c.out + 16 * tile0) * kw + run * kRunWords + lane;
                    for (int r = 0; r < 16 * h; ++r) {
                        const bool there = r < rows_left && run * kRunWords + lane < kw &&
                                           LQ_IN_BOUNDS(((long long)u.e * c.out + 16 * tile0 + r) * kw + run * kRunWords + lane,
                                                        (long long)c.experts * c.out * kw);
                        cp_async4(a_st + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4,
                                  there ? w0 + (long long)r * kw : c.packed, there);
                    }
                }
                const uint32_t u_st = a_st + p.hmax * 2048 + lane * 16;
                const int k_left = c.K - run * kRunK - 8 * lane;  // in 16-byte chunks 256 k apart
#pragma unroll
                for (int i = 0; i < COLS; ++i)
                    if (i < u.slots) {
                        const uint16_t* from = src[i] + run * kRunK;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const bool there = src[i] && 256 * x < k_left &&
                                               LQ_IN_BOUNDS(from - c.u + 256 * x + 7, (long long)c.tokens * c.K);
                            cp_async16(u_st + i * kUPitch + 512 * x, there ? from + 256 * x : c.u, there);
                        }
                    }
                cp_async_arrive(bar);
                last = st, last_phase = phase;
                advance();
            }
        }
        cp_async_wait_all();
        // no TMA copy of this warp is in flight either: its stages are filled in turn, so those before its last
        // one have been waited for by a later wait on their consumers, or are waited for here
        if (TMA && last >= 0)
            for (int back = 0; back < p.stages; back += kProducers) {
                int s = last - back, ph = last_phase;
                if (s < 0) s += p.stages, ph ^= 1;
                mbar_wait(full0 + 8 * s, ph, status);
            }
        return;
    }

    // ---- consumers
    int red_phase = 1;
    const int g = lane >> 2, t = lane & 3, quarter = warp & 3, group = warp >> 2;
    const uint32_t rot = t >= 2 ? 0x1032u : 0x3210u;
    int turn = 0;  // the group that takes the next run
    for (long long unit = blockIdx.x; walk.find<true>(c, COLS, p.nblk, unit, lane, u); unit += gridDim.x) {
        int tile0;
        const int h = block_tiles(p, u.blk, tile0);
        float acc[H][4];
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
        for (int run = 0; run < runs; ++run) {
            if (turn == group) {
                if (!mbar_try_wait(full0 + 8 * st, phase) && !*abort_flag && !mbar_wait(full0 + 8 * st, phase, status))
                    *abort_flag = 1;
                const uint32_t a_st = ring + st * p.stage_bytes;
                const uint32_t u_other = t >= 2 ? -32 : 32;
                // columns past the pass's read zeros (no branch around the loads: it cost 500 clocks a run)
                const uint32_t u_at = (g < u.slots ? a_st + p.hmax * 2048 + g * kUPitch + quarter * 512 + t * 64 : zeros) + (t >= 2 ? 32 : 0);
                uint32_t b[2][16];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t at = u_at + x * 256 + half * 16;
                        const uint4 lo = lds128(at), hi = lds128(at + u_other);
                        const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, v[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            b[x][8 * half + 2 * i] = __byte_perm(l[i], v[i], 0x5410);
                            b[x][8 * half + 2 * i + 1] = __byte_perm(l[i], v[i], 0x7632);
                        }
                    }
                // row g of tile i: chunk 2 quarter + x, swizzled by the row; rows 8 apart share the swizzle
                const uint32_t a_row = a_st + g * 128 + t * 4;
                // Two tiles at a time, so that two chains of accumulation overlap, in steps of 128 k; the words of the
                // next step are loaded ahead. The second tile may be past the block's (words that are in the
                // stage, sums that are not used): a path for single tiles made blocks of odd height 3%
                // faster and the others up to 10% slower.
                auto load_words = [&](uint32_t (&to)[2][2], int i, int x) {
                    const uint32_t at = a_row + i * 2048 + (((2 * quarter + x) ^ g) << 4);
#pragma unroll
                    for (int k = 0; k < 2; ++k) to[k][0] = lds32(at + k * 2048), to[k][1] = lds32(at + k * 2048 + 1024);
                };
                uint32_t w[2][2], next[2][2];
                load_words(next, 0, 0);
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    if (i >= h) break;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            w[k][0] = __byte_perm(next[k][0], 0, rot), w[k][1] = __byte_perm(next[k][1], 0, rot);
                        if (x == 0)
                            load_words(next, i, 1);
                        else if (i + 2 < H)
                            load_words(next, i + 2, 0);
#pragma unroll
                        for (int j = 0; j < 16; j += 2)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                mma_bf16(acc[i + k], sign_pair(w[k][0], p, j), sign_pair(w[k][1], p, j),
                                         sign_pair(w[k][0], p, j + 1), sign_pair(w[k][1], p, j + 1), b[x][j], b[x][j + 1]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * st);
            }
            if (++turn == GROUPS) turn = 0;
            advance();
        }

        // ---- this warp's sums, once the epilogue has read those of the block before
        if (!mbar_try_wait(red_empty, red_phase) && !*abort_flag && !mbar_wait(red_empty, red_phase, status)) *abort_flag = 1;
        red_phase ^= 1;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            if (i >= h) break;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                red[(warp * COLS + 2 * t + (j & 1)) * p.rp + 16 * i + g + (j >> 1) * 8] = acc[i][j];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(red_full);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<EncodeTiledFn>(p)
                   : nullptr;
    }();
    return fn;
}

template <bool TMA>
cudaError_t launch_as(const GroupedCall& c, const Plan& p, int h, unsigned* status, cudaStream_t st, int sms) {
    CUtensorMap maps[2] = {};  // sign words of all experts in boxes of 16 h and 16 (h - 1) rows
    if (TMA) {
        EncodeTiledFn encode = encode_fn();
        if (!encode) return cudaErrorNotSupported;
        cuuint64_t gdim[2] = {(cuuint64_t)(c.K / 32), (cuuint64_t)c.experts * c.out};
        cuuint64_t gstride[1] = {(cuuint64_t)c.K / 8};
        cuuint32_t estride[2] = {1, 1};
        for (int i = 0; i < 2; ++i) {
            cuuint32_t box[2] = {(cuuint32_t)kRunWords, (cuuint32_t)(16 * (h - i > 0 ? h - i : 1))};
            if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint32_t*>(c.packed), gdim, gstride, box, estride,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return cudaErrorInvalidValue;
        }
    }
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(mma_kernel<TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(kSmemMax + 1024));
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    mma_kernel<TMA><<<sms, THREADS, p.smem, st>>>(maps[0], maps[1], c, p, status);
    return cudaGetLastError();
}

// Stages that fit beside blocks of h tiles, in whole rounds of the producers and of the groups: a stage then
// belongs to one of each, which see all its phases (a wait goes by a phase's parity; stages are filled
// and freed out of order, so another stage's phase does not tell).
int ring_stages(const GroupedCall& c, Plan& p, int h) {
    p.hmax = h;
    p.rp = 16 * h + 4;
    const size_t red = (size_t)CONSUMERS * COLS * p.rp * 4;
    const int cols = c.n < COLS ? c.n : COLS;
    p.stage_bytes = (h * 2048 + cols * kUPitch + 1023) / 1024 * 1024;
    const int fit = (int)((kSmemMax - kHead - red) / p.stage_bytes);
    p.stages = (fit > kMaxStages ? kMaxStages : fit) / kProducers * kProducers;
    p.smem = 1024 + (size_t)p.stages * p.stage_bytes + kHead + red;
    return p.stages;
}

}  // namespace

cudaError_t launch_grouped_mma(const GroupedCall& c, unsigned* status, cudaStream_t st, int sms) {
    Plan p{};
    for (int j = 0; j < 16; ++j) p.shift[j] = 1u << (15 - j);
    const int tiles = (c.out + 15) / 16;
    const int active = c.n < c.experts ? c.n : c.experts;  // experts expected to have slots, a pass of columns each
    // Block height: the rounds of blocks over the SMs times their length (a block's fixed cost is about one
    // tile), blocks as many as fill the rounds.
    double best = 0;
    for (int h = 1; h <= H && ring_stages(c, p, h) > 0; ++h) {
        const long long least = (tiles + h - 1) / h, rounds = (active * least + sms - 1) / sms;
        long long nblk = rounds * sms / active;
        nblk = nblk < least ? least : nblk > tiles ? tiles : nblk;
        const double cost = (double)rounds * ((double)tiles / nblk + 1);
        if (best == 0 || cost < best) best = cost, p.nblk = (int)nblk;
    }
    const int h = (tiles + p.nblk - 1) / p.nblk;  // blocks have h or h - 1 tiles
    ring_stages(c, p, h);
    p.low = tiles / p.nblk;
    p.tall = tiles % p.nblk;
    return c.K % 128 == 0 ? launch_as<true>(c, p, h, status, st, sms) : launch_as<false>(c, p, h, status, st, sms);
}

}  // namespace lq

LQ_DEBUG_FLAG_TAKE(debug_take_grouped_mma)
