// Products grouped by expert for many rows per expert (prefill and large batches), on
// tcgen05; lq_grouped.cu routes here.
//
//   z[i][r] = s[r] sum_k sigma[r][k] u[row(i)][k] + bias[r]
//
// A unit is a tile of 128 weight rows by up to BN slots of one expert (256, 128 or 64);
// persistent CTAs (one per SM) take units in turn. The MMA's width N is the tile's slots
// rounded up to 16, so a short tail of an expert costs what it needs. K is walked in
// steps of 64 (128 for the narrowest tiles) through a ring of stages. Roles:
//   warp 0        u rows of the slots by TMA (128-byte swizzle)
//   warp 1        issues the MMAs (M = 128, K = 16, bf16, fp32 in TMEM); narrow tiles: warp 14 too
//   warps 2..9    two groups that fill the stages in turn; a thread owns one weight row, loads its sign
//                 words well ahead and stores them as bf16 +-1 into the stage in the swizzled layout
//   warps 10..13  epilogue of the tile before, from the other of two accumulators: scale, bias,
//                 activation or gate, residual, one rounding, store. A thread owns one weight
//                 row, so a warp stores 32 neighbouring outputs.
// With `rows`, a kernel before it copies the slots' rows of u into the workspace: gathering
// them in this kernel, four to a TMA instruction, took 1200 clocks per 64 k of 256 slots
// (the MMAs take 512), and with cp.async 1900; the copy costs n K bytes written and read.
// Few tiles of a single layer are cut along K, so that they fill the SMs (plan_split). Products are exact; only the
// fp32 sums round. Every wait is bounded.
//
// What bounds it. Wide tiles: the tensor cores under the power cap (13824 x 12288, 2048 tokens, gated:
// 427 us = 1630 TFLOP/s in short bursts, 499 us = 1394 of the 1434 TFLOP/s that the library's product
// sustains). Narrow ones: no unit is saturated. Of a CTA's active time at 64 tokens the tensor pipe works 31%, the ALU
// pipe (the expansion) 53%, and both sides of shared memory run at less than the rates that wide tiles reach (the
// stores of signs and u 58 against 70%, the MMAs' reads 46 against 65%); a step of 128 k takes 740 clocks, which are
// waits of the roles for one another and for sign words on their way (38 us warm, 44 with the signs from HBM; 128
// tokens 54 and 58). And 108 tiles leave a quarter of the SMs idle. Which of the waits is the longest is not known.
#include <cuda.h>

#include "lq_debug.cuh"
#include "lq_epilogue.cuh"
#include "lq_grouped.cuh"
#include "lq_internal.h"
#include "lq_sm100.cuh"

namespace lq {
namespace {

using namespace sm100;

constexpr int BM = 128, BK = 64;        // BK: k of one swizzled tile
constexpr int A_TILE = BM * BK * 2;
constexpr int kBox = 64;  // rows of a tiled load of u of a short tile; a long one loads all BN rows at once
constexpr int UNPACK_WARP = 2, EPILOGUE_WARP = 10, ISSUER_WARP = 14;

// A stage is SUB tiles of 64 k. A thread that issues a stage's MMAs spends ~400 clocks more on its commit and
// on the next wait, which the MMAs of a narrow tile do not cover: there the stages alternate between two
// issuing warps, each with accumulators of its own, added in the epilogue (64 tokens of 13824 x 12288:
// 46 -> 38 us), and the narrowest tiles commit every 128 k (64 k steps of N = 64 took one issuer 500
// clocks each, of which the MMAs 190).
//
// A wait goes by a phase's parity, so whoever waits on a stage has to know that the phase before is over, and
// stages are freed and filled out of order. So every stage belongs to one unpack group and one issuer, by its
// number's parity (rings have an even number of stages), which see all its phases; the loads of u and a single
// issuer see all phases of all stages.
template <int BN>
struct Ring {
    static constexpr int ISSUERS = BN == 256 ? 1 : 2, THREADS = 32 * (ISSUER_WARP + ISSUERS - 1);
    static constexpr int SUB = BN == 64 ? 2 : 1;
    static constexpr int STAGES = BN == 128 ? 6 : 4;
    static_assert(STAGES % 2 == 0, "a stage has one unpack group and one issuer");
    static constexpr int A_STAGE = SUB * A_TILE, B_TILE = BN * BK * 2, B_STAGE = SUB * B_TILE;
    static constexpr size_t SMEM_BYTES = 1024 + STAGES * (A_STAGE + B_STAGE) + 256;
};

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// One lane of a converged warp, in the form that lets the compiler keep the operands of
// the instructions behind it in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// 16 sign bits (in the low half of x) as eight bf16 pairs: pair i holds bits 2i and 2i + 1.
__device__ __forceinline__ void expand16(uint32_t x, uint32_t* v) {
    const uint32_t q = (x & 0x5555u) | ((x & 0xAAAAu) << 15);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t y = q << (15 - 2 * i);
        asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(v[i]) : "r"(y), "r"(0x80008000u), "r"(0xBF80BF80u));  // (y & b) ^ c
    }
}

// N outputs of one weight row: element at + j * width of o, for slots j below count, with the residual.
// Every choice is made outside the loops over j: a warp works alone on its scheduler here, and
// branches between the elements cost it 330 clocks an element (45 us for a tile of 256 slots).
template <int N, bool BF16>
__device__ __forceinline__ void store_row(const GroupedCall& c, float (&y)[N], long long at, int width, int count) {
    using T = typename Elem<BF16>::T;
    const long long extent = (long long)c.n * width;
    (void)extent;
    T* o = static_cast<T*>(c.o) + at;
    if (c.residual) {
        const T* res = static_cast<const T*>(c.residual) + at;
        T r[N];
#pragma unroll
        for (int j = 0; j < N; ++j) r[j] = j < count && LQ_IN_BOUNDS(at + (long long)j * width, extent) ? __ldg(res + (long long)j * width) : T(0);
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] += Elem<BF16>::to_float(r[j]);
    }
    if (count >= N) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (LQ_IN_BOUNDS(at + (long long)j * width, extent)) o[(long long)j * width] = Elem<BF16>::from_float(y[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < count && LQ_IN_BOUNDS(at + (long long)j * width, extent))
                o[(long long)j * width] = Elem<BF16>::from_float(y[j]);
    }
}

// One row's outputs for 32 slots of the tile, from its accumulator columns.
template <bool BF16>
__device__ __forceinline__ void store_chunk(const GroupedCall& c, float (&z)[32], int m, int width, int slot0, int count,
                                            int lane) {
    if (!c.glu) {
        activate_all(z, c.act);
        if (m < c.out) store_row<32, BF16>(c, z, (long long)slot0 * width + m, width, count);
        return;
    }
    // gate rows are the even lanes', the other factors the odd lanes': lane pairs swap
    // halves, the even lane finishes slots 0..15 and the odd lane slots 16..31
    const bool odd = lane & 1;
    float gate[16], up[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float own = odd ? z[16 + j] : z[j], other = __shfl_xor_sync(0xffffffffu, odd ? z[j] : z[16 + j], 1);
        gate[j] = odd ? other : own;
        up[j] = odd ? own : other;
    }
    activate_all(gate, c.act);
#pragma unroll
    for (int j = 0; j < 16; ++j) gate[j] *= up[j];
    const int j0 = odd ? 16 : 0;
    if (m < c.out) store_row<16, BF16>(c, gate, (long long)(slot0 + j0) * width + m / 2, width, count - j0);
}

// A layer's tiles cut along K, when they are too few or too uneven for the SMs (plan_split). A part's epilogue
// warps write its sums to `part`; of a tile's parts, the warp that counts itself last adds them, in the order of
// k whoever that is, and stores the outputs.
struct Split {
    int parts;
    unsigned* count;  // [tiles][4 warps], cleared by the kernel before
    float4* part;     // [tiles][parts][BN / 4][128], four slots each
};

__global__ void __launch_bounds__(256) clear_kernel(uint4* to, int n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the products may start meanwhile
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) to[i] = make_uint4(0, 0, 0, 0);
}

// BN: slots of a full tile. SPLIT: tiles are cut along K. VEC: K a multiple of 128, so that rows of sign words are
// 16-byte aligned.
template <int BN, bool VEC, bool SPLIT>
__global__ void __launch_bounds__(Ring<BN>::THREADS, 1)
    tc_kernel(const __grid_constant__ CUtensorMap tmap_u, const __grid_constant__ CUtensorMap tmap_all,
              const __grid_constant__ GroupedCall c, const Split split, unsigned* status) {
    constexpr int STAGES = Ring<BN>::STAGES, SUB = Ring<BN>::SUB, A_STAGE = Ring<BN>::A_STAGE;
    constexpr int B_STAGE = Ring<BN>::B_STAGE, B_TILE = Ring<BN>::B_TILE, STEP = SUB * BK;
    constexpr int ISSUERS = Ring<BN>::ISSUERS, ACC = ISSUERS * BN;  // columns of a tile's accumulators
    extern __shared__ uint8_t smem_raw[];
    // 1024-byte aligned for the 128-byte swizzle
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sA = smem_addr(smem), sB = sA + STAGES * A_STAGE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * (A_STAGE + B_STAGE));
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * STAGES;
    const uint32_t acc_full0 = empty0 + 8 * STAGES, acc_empty0 = acc_full0 + 16, drained = acc_empty0 + 16;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kw = c.K >> 5, steps = (c.K + STEP - 1) / STEP, nblk = (c.out + BM - 1) / BM;

    if (threadIdx.x == 0) {
        for (int st = 0; st < STAGES; ++st) {
            mbar_init(full0 + 8 * st, 1 + 128);
            mbar_init(empty0 + 8 * st, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(acc_full0 + 8 * a, ISSUERS);
            mbar_init(acc_empty0 + 8 * a, 128);
        }
        mbar_init(drained, ISSUERS);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmap_u);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 2 * ACC);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // A role gives up when a wait of its own runs out or another role has given up;
    // the decision is one for the whole warp, which walks the units together.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const bool ok = !*abort_flag && mbar_wait(bar, parity, status);
        if (__all_sync(0xffffffffu, ok)) return true;
        *abort_flag = 1;
        return false;
    };

    UnitWalk walk;
    Unit u;
    long long tile;              // the unit's tile, and its range of steps: [kb0, kb0 + nkb)
    int part = 0, kb0 = 0, nkb = steps;
    auto next = [&](long long unit) {
        tile = unit;
        if constexpr (SPLIT) {
            tile = unit / split.parts;
            part = (int)(unit - tile * split.parts);
            kb0 = (int)((long long)part * steps / split.parts);
            nkb = (int)((long long)(part + 1) * steps / split.parts) - kb0;
        }
        return walk.find<false>(c, BN, nblk, tile, lane, u);
    };
    int st = 0, phase = 0;  // ring position, kept by each role
    auto advance = [&] {
        if (++st == STAGES) st = 0, phase ^= 1;
    };
    bool go = true;
    // The same for a role's next stage, with the poll before the work on the current one: after a commit
    // a poll takes hundreds of clocks, which would come between the MMAs of two stages. poll() looks at the
    // stage after this one, ready() waits for the current stage unless the last poll saw it complete.
    bool seen = false;
    auto poll = [&](uint32_t bar0, uint32_t flip) {
        const int st1 = st + 1 == STAGES ? 0 : st + 1;
        seen = mbar_try_wait(bar0 + 8 * st1, (st1 ? phase : phase ^ 1) ^ flip);
    };
    auto ready = [&](uint32_t bar0, uint32_t flip) {
        const bool known = __all_sync(0xffffffffu, seen);
        seen = false;
        return known || wait(bar0 + 8 * st, phase ^ flip);
    };
    if (warp == 0) {
        // ---- u tiles
        int issued = 0;
        for (long long unit = blockIdx.x; go && next(unit); unit += gridDim.x) {
            const bool all = u.slots > BN - kBox;
            const int boxes = all ? BN / kBox : (u.slots + kBox - 1) / kBox;
            for (int kb = 0; kb < nkb; ++kb) {
                if (!(go = ready(empty0, 1))) break;
                poll(empty0, 1);
                if (elect_one()) {
                    const uint32_t dst = sB + st * B_STAGE, bar = full0 + 8 * st;
                    mbar_arrive_expect_tx(bar, SUB * boxes * kBox * 128);
#pragma unroll
                    for (int x = 0; x < SUB; ++x) {
                        const uint32_t to = dst + x * B_TILE;
                        if (all)
                            tma_load_2d(to, &tmap_all, (kb0 + kb) * STEP + x * BK, u.slot0, bar);
                        else
                            for (int i = 0; i < boxes; ++i)
                                tma_load_2d(to + i * kBox * 128, &tmap_u, (kb0 + kb) * STEP + x * BK, u.slot0 + i * kBox, bar);
                    }
                }
                __syncwarp();
                ++issued;
                advance();
            }
        }
        // leave no copy in flight: the last load of each stage has landed
        for (int back = issued < STAGES ? issued : STAGES; back > 0; --back) {
            const int at = issued - back;
            mbar_wait(full0 + 8 * (at % STAGES), (at / STAGES) & 1, status);
        }
    } else if (warp == 1 || warp >= ISSUER_WARP) {
        // ---- MMAs: of two issuers, each takes every other stage
        const int issuer = warp == 1 ? 0 : 1;
        int acc = 0, acc_phase = 0;
        const uint64_t a_desc = smem_desc_sw128(sA), b_desc = smem_desc_sw128(sB);
        for (long long unit = blockIdx.x; go && next(unit); unit += gridDim.x) {
            const uint32_t idesc = idesc_bf16_f32(BM, (u.slots + 15) / 16 * 16);
            if (!(go = wait(acc_empty0 + 8 * acc, acc_phase ^ 1))) break;
            tc_fence_after();
            const uint32_t to = tmem + acc * ACC + issuer * BN;
            bool first = true;  // the issuer's first stage of the tile
            for (int kb = 0; kb < nkb; ++kb) {
                if (st % ISSUERS == issuer) {
                    if (ISSUERS == 1) {
                        if (!(go = ready(full0, 0))) break;
                        poll(full0, 0);
                    } else if (!(go = wait(full0 + 8 * st, phase))) {
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        // 16 k are 32 bytes of a swizzled row, 2 in the descriptor's address field
                        const uint64_t a = a_desc + (uint32_t)st * (A_STAGE >> 4), b = b_desc + (uint32_t)st * (B_STAGE >> 4);
#pragma unroll
                        for (int x = 0; x < SUB; ++x)
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk)
                                umma_f16(to, a + x * (A_TILE >> 4) + 2 * kk, b + x * (B_TILE >> 4) + 2 * kk, idesc,
                                         !first || (x | kk) != 0);
                        umma_commit(empty0 + 8 * st);
                    }
                    __syncwarp();
                    first = false;
                }
                advance();
            }
            if (!go) break;
            if (elect_one()) umma_commit(acc_full0 + 8 * acc);  // arrives at once if no stage of the tile was its own
            __syncwarp();
            if (++acc == 2) acc = 0, acc_phase ^= 1;
        }
        if (elect_one()) umma_commit(drained);  // no MMA is in flight when TMEM is freed (the issuing lane is always the same)
        __syncwarp();
        mbar_wait(drained, 0, status);
    } else if (warp < EPILOGUE_WARP) {
        // ---- signs: each of two groups fills every other stage
        constexpr int WORDS = 2 * SUB, AHEAD = 16 / WORDS;  // sign words of a row and stage; stages loaded ahead
        const int group = (warp - UNPACK_WARP) >> 2, row = (threadIdx.x - 32 * UNPACK_WARP) & 127;
        const uint32_t row_off = (row >> 3) * 1024 + (row & 7) * 128, sw = row & 7;
        for (long long unit = blockIdx.x; go && next(unit); unit += gridDim.x) {
            const int r = min(u.blk * BM + row, c.out - 1);  // rows past `out` are computed but not stored
            // Past the row's end its last words are read again: u is zero there. (No branch: a load merged with
            // another value would be waited for at once.)
            const uint32_t* w0 = c.packed + ((long long)u.e * c.out + r) * kw;
            auto words_there = [&](int x, int count) {  // `count` words from word x of the row
                return LQ_IN_BOUNDS(w0 - c.packed + x, (long long)c.experts * c.out * kw - count + 1);
            };
            auto load = [&](int kb, uint32_t (&to)[WORDS]) {
                const int x = WORDS * (kb0 + kb);
                if constexpr (VEC && SUB == 2) {
                    if (!words_there(min(x, kw - 4), 4)) return;
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(w0 + min(x, kw - 4)));
                    to[0] = v.x, to[1] = v.y, to[2] = v.z, to[WORDS - 1] = v.w;
                } else if constexpr (VEC) {
                    if (!words_there(min(x, kw - 2), 2)) return;
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(w0 + min(x, kw - 2)));
                    to[0] = v.x, to[1] = v.y;
                } else {
#pragma unroll
                    for (int i = 0; i < WORDS; ++i)
                        if (words_there(min(x + i, kw - 1), 1)) to[i] = __ldg(w0 + min(x + i, kw - 1));
                }
            };
            const int st0 = st, phase0 = phase;  // ring position of the unit's first stage
            const int begin = (group ^ st0) & 1;
            uint32_t ahead[AHEAD][WORDS];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) load(begin + 2 * i, ahead[i]);
            for (int kb1 = begin; kb1 < nkb && go; kb1 += 2 * AHEAD) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int kb = kb1 + 2 * i;
                    if (kb >= nkb || !go) break;
                    uint32_t w[WORDS];
#pragma unroll
                    for (int x = 0; x < WORDS; ++x) w[x] = ahead[i][x];
                    load(kb + 2 * AHEAD, ahead[i]);
                    const int at = st0 + kb, s = at % STAGES, ph = phase0 ^ ((at / STAGES) & 1);
#pragma unroll
                    for (int half = 0; half < SUB; ++half) {
                        uint32_t v[32];
                        expand16(w[2 * half], v);
                        expand16(w[2 * half] >> 16, v + 8);
                        expand16(w[2 * half + 1], v + 16);
                        expand16(w[2 * half + 1] >> 16, v + 24);
                        if (half == 0)
                            if (!(go = wait(empty0 + 8 * s, ph ^ 1))) break;
                        const uint32_t dst = sA + s * A_STAGE + half * A_TILE + row_off;
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            st_shared_v4(dst + ((q ^ sw) << 4), v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    }
                    if (!go) break;
                    fence_proxy_async_smem();
                    mbar_arrive(full0 + 8 * s);
                }
            }
            st = st0 + nkb;
            phase = phase0 ^ ((st / STAGES) & 1);
            st %= STAGES;
        }
    } else {
        // ---- epilogue: a warp may only reach its own quarter of the TMEM lanes (warp % 4)
        const int q = warp & 3, width = c.glu ? c.out / 2 : c.out;
        int acc = 0, acc_phase = 0, issuer0 = 0;  // issuer0: the issuer of the unit's first stage
        const long long tiles = (long long)nblk * ((c.n + BN - 1) / BN), parts_extent = tiles * split.parts * (BN / 4) * BM;
        (void)parts_extent;
        if constexpr (SPLIT) asm volatile("griddepcontrol.wait;" ::: "memory");  // the counts are cleared
        auto finish = [&](float (&z)[32], int c0, float sr, float br, int m) {
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = fmaf(sr, z[j], br);
            if (c.o_bf16)
                store_chunk<true>(c, z, m, width, u.slot0 + c0, u.slots - c0, lane);
            else
                store_chunk<false>(c, z, m, width, u.slot0 + c0, u.slots - c0, lane);
        };
        for (long long unit = blockIdx.x; go && next(unit); unit += gridDim.x) {
            const int m = u.blk * BM + q * 32 + lane;
            const long long at = (long long)u.e * c.out + min(m, c.out - 1);
            const float sr = __ldg(c.s + at), br = c.bias ? __ldg(c.bias + at) : 0.f;
            if (!(go = wait(acc_full0 + 8 * acc, acc_phase))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < u.slots; c0 += 32) {
                uint32_t v[32];
                const uint32_t from = tmem + acc * ACC + ((uint32_t)(q * 32) << 16) + c0;
                tmem_ld_32x32b_x32(from + issuer0 * BN, v);
                tmem_ld_wait();
                float z[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(v[j]);
                if (ISSUERS == 2 && nkb > 1) {
                    tmem_ld_32x32b_x32(from + (issuer0 ^ 1) * BN, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) z[j] += __uint_as_float(v[j]);
                }
                if constexpr (SPLIT) {
                    float4* to = split.part + ((tile * split.parts + part) * BN + c0) / 4 * BM + q * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        if (c0 + j < u.slots && LQ_IN_BOUNDS(to + j / 4 * BM - split.part, parts_extent))
                            __stcg(to + j / 4 * BM, make_float4(z[j], z[j + 1], z[j + 2], z[j + 3]));
                } else {
                    finish(z, c0, sr, br, m);
                }
            }
            tc_fence_before();
            mbar_arrive(acc_empty0 + 8 * acc);
            if constexpr (SPLIT) {
                __threadfence();  // the sums are there before the count says so
                __syncwarp();
                unsigned before = 0;
                if (lane == 0 && LQ_IN_BOUNDS(tile, tiles)) before = atomicAdd(split.count + tile * 4 + q, 1u);
                if (__shfl_sync(0xffffffffu, before, 0) == split.parts - 1u) {
                    __threadfence();
#pragma unroll 1
                    for (int c0 = 0; c0 < u.slots; c0 += 32) {
                        const float4* from = split.part + (tile * split.parts * BN + c0) / 4 * BM + q * 32 + lane;
                        float z[32] = {};
#pragma unroll 2
                        for (int x = 0; x < split.parts; ++x, from += BN / 4 * BM) {
                            float4 v[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                v[j] = c0 + 4 * j < u.slots && LQ_IN_BOUNDS(from + j * BM - split.part, parts_extent)
                                           ? __ldcg(from + j * BM)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                z[4 * j] += v[j].x, z[4 * j + 1] += v[j].y, z[4 * j + 2] += v[j].z, z[4 * j + 3] += v[j].w;
                        }
                        finish(z, c0, sr, br, m);
                    }
                }
            }
            if (ISSUERS == 2) issuer0 ^= nkb & 1;
            if (++acc == 2) acc = 0, acc_phase ^= 1;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * ACC);
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

// Slot i's row of u, zeros for a row outside it; slots of no expert are left as they are.
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ GroupedCall c, uint4* __restrict__ dst) {
    const int chunks = c.K / 8;
    const int end = min(max(__ldg(c.offsets + c.experts), 0), c.n);
    for (int i = blockIdx.x; i < end; i += gridDim.x) {
        const int row = __ldg(c.rows + i);
        const bool there = row >= 0 && row < c.tokens;
        const uint4* src = reinterpret_cast<const uint4*>(c.u) + (there ? (long long)row * chunks : 0);
        for (int x = threadIdx.x; x < chunks; x += 256) {
            uint4 v = {0, 0, 0, 0};
            if (there && LQ_IN_BOUNDS((long long)row * chunks + x, (long long)c.tokens * chunks)) v = __ldg(src + x);
            if (LQ_IN_BOUNDS((long long)i * chunks + x, (long long)c.n * chunks)) dst[(long long)i * chunks + x] = v;
        }
    }
}

template <int BN, bool VEC, bool SPLIT>
cudaError_t launch_as(const GroupedCall& c, const Split& split, unsigned* status, cudaStream_t st, int sms) {
    EncodeTiledFn encode = encode_fn();
    if (!encode) return cudaErrorNotSupported;
    CUtensorMap map, map_all;  // u in boxes of kBox and of BN rows
    cuuint64_t gdim[2] = {(cuuint64_t)c.K, (cuuint64_t)c.tokens};
    cuuint64_t gstride[1] = {(cuuint64_t)c.K * 2};
    cuuint32_t estride[2] = {1, 1};
    for (int i = 0; i < 2; ++i) {
        cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)(i ? BN : kBox)};
        if (encode(i ? &map_all : &map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(c.u), gdim, gstride, box,
                   estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(tc_kernel<BN, VEC, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)Ring<BN>::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms);
    cfg.blockDim = dim3(Ring<BN>::THREADS);
    cfg.dynamicSmemBytes = Ring<BN>::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = SPLIT ? 1 : 0;  // behind clear_kernel alone, which is launched when all before it is complete
    return cudaLaunchKernelEx(&cfg, tc_kernel<BN, VEC, SPLIT>, map, map_all, c, split, status);
}

template <int BN>
cudaError_t launch_bn(const GroupedCall& c, const Split& split, unsigned* status, cudaStream_t st, int sms) {
    if (split.parts > 1)
        return c.K % 128 == 0 ? launch_as<BN, true, true>(c, split, status, st, sms) : launch_as<BN, false, true>(c, split, status, st, sms);
    return c.K % 128 == 0 ? launch_as<BN, true, false>(c, split, status, st, sms) : launch_as<BN, false, false>(c, split, status, st, sms);
}

int tile_slots(int each) { return each <= 64 ? 64 : each <= 128 ? 128 : 256; }

// Parts along K of each tile of one layer: the rounds over the SMs times a part's steps and its own cost in steps
// (its sums written and counted, all parts' read by the last, 4 to 20 us). us whole and in parts: 4096 x 10240 at 64 tokens 36
// and 19.6 (4 parts), at 128 52 and 27, at 512 65 and 48; 11007 x 9728 at 61 tokens 37 and 44 (5 parts, not taken),
// 13824 x 12288 at 256 71 and 101 (4 parts, not taken). Three rounds of parts bound the workspace.
int plan_split(const GroupedCall& c, int bn, long long& tiles) {
    constexpr int kSms = 148;
    const int step = bn == 64 ? 128 : 64;
    const double wide = bn == 64 ? 1 : bn == 128 ? 2 : 3.2;
    const int steps = (c.K + step - 1) / step;
    tiles = (long long)((c.out + BM - 1) / BM) * (((long long)c.n + bn - 1) / bn);
    if (c.offsets || tiles >= 2 * kSms) return 1;
    int best = 1;
    double cost = 0.95 * ((tiles + kSms - 1) / kSms) * steps;
    for (int parts = 2; parts <= 16 && parts <= steps && parts * tiles <= 3 * kSms; ++parts) {
        const double with = (double)((tiles * parts + kSms - 1) / kSms) * ((steps + parts - 1) / parts + wide * (6 + 2.75 * parts));
        if (with < cost) cost = with, best = parts;
    }
    return best;
}

size_t count_bytes(long long tiles) { return ((size_t)tiles * 16 + 255) / 256 * 256; }

}  // namespace

size_t grouped_tc_workspace_size(const GroupedCall& c, int each) {
    if (c.offsets) return c.rows ? (size_t)c.n * c.K * 2 : 0;  // the copied rows
    long long tiles;
    const int bn = tile_slots(each), parts = plan_split(c, bn, tiles);
    return parts > 1 ? count_bytes(tiles) + (size_t)tiles * parts * bn * BM * 4 : 0;
}

cudaError_t launch_grouped_tc(const GroupedCall& call, void* ws, unsigned* status, cudaStream_t st, int sms, int each) {
    GroupedCall c = call;
    if (c.rows) {
        gather_kernel<<<c.n < 8 * sms ? c.n : 8 * sms, 256, 0, st>>>(c, static_cast<uint4*>(ws));
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        c.u = static_cast<const uint16_t*>(ws);
        c.tokens = c.n;
        c.rows = nullptr;
    }
    const int bn = tile_slots(each);
    long long tiles;
    Split split{plan_split(c, bn, tiles), nullptr, nullptr};
    if (split.parts > 1) {
        split.count = static_cast<unsigned*>(ws);
        split.part = reinterpret_cast<float4*>(static_cast<uint8_t*>(ws) + count_bytes(tiles));
        clear_kernel<<<(unsigned)((tiles + 255) / 256), 256, 0, st>>>(static_cast<uint4*>(ws), (int)tiles);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (bn == 64) return launch_bn<64>(c, split, status, st, sms);
    if (bn == 128) return launch_bn<128>(c, split, status, st, sms);
    return launch_bn<256>(c, split, status, st, sms);
}

}  // namespace lq

LQ_DEBUG_FLAG_TAKE(debug_take_grouped_tc)
